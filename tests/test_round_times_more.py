"""The timing tool over both files of cases: the work of the inputs that are run, and names of kernels with switches among their
template arguments."""

import pytest
import torch

from gated_deltanet_speculative_amd import round_times as T


@pytest.mark.parametrize("more", [False, True])
def test_work_is_that_of_the_inputs(more):
    """Two chunks, lengths 16384 and 12288, nodes 2048 and 1536: the pairs by hand, with either length under either count."""
    ops = T.operators(more)
    case = next(c for c in ops.listed() if c["name"] == "attn chunk 2x2048 16k")
    state = lambda *lens: dict(len=torch.tensor([5, lens[1], 7, lens[0]]), slots=torch.tensor([3, 1], dtype=torch.int32))  # noqa: E731
    same, other = [(2048, 16384), (1536, 12288)], [(2048, 12288), (1536, 16384)]
    flops = lambda lanes: 4.0 * 256 * 16 * sum(n * x + n * (n + 1) / 2 for n, x in lanes)  # noqa: E731
    assert T.work_of(ops, case, [state(16384, 12288)]) == ops.work(case) and ops.work(case)["flops"] == flops(same)
    assert T.work_of(ops, case, [state(12288, 16384)]) == dict(ops.work(case), flops=flops(other))
    assert T.work_of(ops, case, [state(16384, 12288), state(12288, 16384)])["flops"] == (flops(same) + flops(other)) / 2
    for c in ops.listed():
        if not (c["op"] == "attn" and c["ragged"]):
            assert T.work_of(ops, c, []) == ops.work(c)


def test_further_cases_are_complete():
    ops = T.operators(True)
    got = T.cases(ops, further=True)
    assert len({c["name"] for c in got}) == len(got) == len(ops.listed()) + len(T.FURTHER_MORE)
    keys = {c["op"]: set(c) for c in ops.listed()}
    for c in T.FURTHER_MORE:
        assert set(c) - {"rows"} == keys[c["op"]] and ops.work(c)["bytes"] > 0, c["name"]


def test_names_of_kernels_with_switches():
    assert T.kernel_of("_ZN3gdn12_GLOBAL__N_116attn_pair_kernelIDF16bLb1EEEvNS_8AttnArgsENS_8AttnPlanE") == "attn_pair_kernel<bf16, true>"
    assert T.kernel_of("_ZN3gdn12_GLOBAL__N_116attn_rows_kernelIDF16_Li128ELi64ELb0EEEvNS_8AttnArgsENS_8AttnPlanE") == \
        "attn_rows_kernel<f16, 128, 64, false>"
    assert T.kernel_of("void gdn::(anonymous namespace)::attn_few_kernel<float, 64, true>(gdn::AttnArgs, gdn::AttnPlan)") == \
        "attn_few_kernel<float, 64, true>"
    assert T.kernel_of("void gdn::(anonymous namespace)::kv_commit_kernel<0>(gdn::AttnDims, int)") == "kv_commit_kernel<0>"
    misread = "void gdn::(anonymous namespace)::{}_kernel<bool _Accum, {}>(gdn::LogitArgs)"
    assert T.kernel_of(misread.format("adjust_logits", "2")) == "adjust_logits_kernel<bf16, float, 2>"
    assert T.kernel_of(misread.format("attn_pair", "bool, E")) == "attn_pair_kernel<bf16, true>"
