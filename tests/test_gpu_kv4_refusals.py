"""Refusals of the calls over a 4-bit cache and of the logits' rules, argument by argument: the error names the argument, or is
the C call's own code where the sizes are sound for the binding, and nothing that the call could write has changed."""

import collections
import re

import pytest
import torch

import gated_deltanet_speculative_amd as gdn
from test_gpu_kv4_binding import BF, I32, NEEDED, _calls

pytestmark = pytest.mark.gpu
FILL = -7.0

# (call, argument, kind of change): what is refused instead of the argument by its name.  A tensor that gives a size
# (inv_freq: rot_dim / 2; positions: the axes) makes the one that has to fit it the odd one, or is refused by the C call.
OTHER = {("rope", "inv_freq", "empty"): "pair_axis", ("rope", "inv_freq", "longer"): "pair_axis", ("rope", "positions", "empty"): None}
KINDS = {"type": lambda t: t.to(torch.int16), "host": lambda t: t.cpu(), "text": lambda t: "text", "empty": lambda t: t[..., :0],
         "axis": lambda t: t.unsqueeze(0), "longer": lambda t: torch.cat([t, t[:1]]),
         "turned": lambda t: t.transpose(0, -1) if t.dim() > 1 else torch.stack([t, t], -1)[..., 0] if t.numel() > 1 else t.expand(2),
         "None": lambda t: None}
CACHE_KINDS = {"shorter": lambda y: y[..., :-1], "type": lambda y: y.to(I32), "host": lambda y: y.cpu(), "None": lambda y: None,
               "turned": lambda y: y.transpose(-2, -3)}


def _tensors(kw):
    """Every tensor of the arguments, those of the caches among them, by name."""
    out = {}
    for name, t in kw.items():
        if isinstance(t, tuple):
            out |= {f"{name}.{f}": x for f, x in zip(t._fields, t)}
        elif isinstance(t, torch.Tensor):
            out[name] = t
    return out


@pytest.mark.parametrize("call", ["rope", "attn", "commit", "read", "logits"])
def test_a_refusal_names_its_argument_and_writes_nothing(call):
    f, sh, kw = _calls()[call]
    for name in ("q_out", "out", "k_out", "v_out", "workspace"):
        if name in kw:
            kw[name].fill_(FILL)
    for name in ("new_len", "status"):
        if name in kw:
            kw[name].zero_()
    before = {n: t.clone() for n, t in _tensors(kw).items()}
    bits = lambda t: t.contiguous().view(torch.uint8)  # noqa: E731

    def refused(name, what, **other):
        """name: in the error's text; None: the C call's code."""
        with pytest.raises(gdn.GdnError if name is None else (TypeError, ValueError)) as e:
            f(sh, **{**kw, **other})
        assert name is None or re.search(rf"(^|\W){re.escape(name)}(\W|$)", str(e.value)), f"{what}: {e.value}"

    for name, t in kw.items():
        if name in ("cache", "caches"):
            for j, field in enumerate(("k", "k_scale", "v", "v_scale")):
                for kind, change in CACHE_KINDS.items():
                    refused(f"cache.{field}", f"{name}.{field} {kind}", **{name: type(t)(*(change(y) if i == j else y for i, y in enumerate(t)))})
            for other in (t.k, t[:3], 5):
                refused("caches" if name == "caches" and isinstance(other, int) else "cache", f"{name} {type(other)}", **{name: other})
            if name == "caches":
                refused("0 layers", "no layers", caches=[])
                refused("65 layers", "too many layers", caches=[gdn.Kv4Cache(*(y[0] for y in t))] * 65)
                refused("cache.k", "two caches of two layers", caches=[t, t])
            continue
        for kind, change in KINDS.items():
            if kind == "None" and name not in NEEDED[call] or name == "workspace" and kind in ("axis", "longer", "empty"):
                continue
            refused(OTHER.get((call, name, kind), name), f"{name} {kind}", **{name: change(t)})
    if call == "logits":
        refused(None, "workspace too small", workspace=kw["workspace"][:-1])
    torch.cuda.synchronize()
    for n, t in _tensors(kw).items():
        assert torch.equal(bits(t), bits(before[n])), f"{n} was written by a refused call"


def test_caches_of_a_read_without_outputs():
    """The rows that the call allocates are those of the caches' layers; what is no cache of layers is refused by its name."""
    f, sh, kw = _calls()["read"]
    kw.pop("k_out"), kw.pop("v_out")
    t = kw["caches"]
    want = f(sh, **kw)[:2]
    for same in (tuple(t), [gdn.Kv4Cache(*(y[l] for y in t)) for l in range(2)], tuple(gdn.Kv4Cache(*(y[l] for y in t)) for l in range(2)),
                 collections.deque(gdn.Kv4Cache(*(y[l] for y in t)) for l in range(2))):
        assert all(torch.equal(a, b) for a, b in zip(f(sh, **{**kw, "caches": same})[:2], want))
    four = gdn.Kv4Cache(*(torch.cat([y, y]) for y in t))
    got = f(sh, **{**kw, "caches": tuple(gdn.Kv4Cache(*(y[l] for y in four)) for l in range(4))})[:2]
    assert all(torch.equal(a, b) for a, b in zip(got, f(sh, **{**kw, "caches": four})[:2]))
    one = gdn.Kv4Cache(*(y[0] for y in t))
    for bad, name in ((t._replace(k=None), "cache.k"), (one, "cache.k"), (t._replace(v=None), "cache.v"), ([one, t], "cache.k"), (None, "caches")):
        with pytest.raises((TypeError, ValueError), match=re.escape(name)):
            f(sh, **{**kw, "caches": bad})
