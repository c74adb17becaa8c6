"""The timing tool's cases: each of them complete, drawn ones the same for the same seed."""

from gated_deltanet_speculative_amd import round_times as T


def test_cases_are_complete():
    ops = T.operators()
    got = T.cases(ops, further=True, draws=20, seed=3)
    assert len({c["name"] for c in got}) == len(got) == len(ops.listed()) + len(T.FURTHER) + 20
    assert got[-20:] == T.cases(ops, draws=20, seed=3)[-20:] != T.cases(ops, draws=20, seed=4)[-20:]
    keys = {c["op"]: set(c) for c in ops.listed()}
    for c in got:
        assert ops.work(c)["bytes"] > 0
    for c in T.FURTHER:
        assert set(c) - {"rows"} >= keys[c["op"]], c["name"]
    assert [c["name"] for c in T.cases(ops, only="prompt")] == [c["name"] for c in ops.listed() if "prompt" in c["name"]]


def test_summary_groups_dispatches_by_case(tmp_path):
    def table(name, column, rows):
        path = tmp_path / name
        path.write_text("Dispatch_Id,Kernel_Name,Start_Timestamp,End_Timestamp,Counter_Value\n" + "".join(
            f'{i},"{k}",1000,{1000 + v if column else 1000},{0 if column else v}\n' for i, (k, v) in enumerate(rows)))
        return str(path)

    few = "void gdn::(anonymous namespace)::attn_few_kernel<float, 64>(gdn::AttnArgs, gdn::AttnPlan)"
    join = "_ZN3gdn12_GLOBAL__N_116attn_join_kernelIDF16bLi64EEEvNS_8AttnArgsENS_8AttnPlanE"
    fill = "void at::native::fill(int)"
    rows = [(fill, 1), (few, 4000), (join, 1000), (few, 6000), (join, 3000), (few, 5000), (join, 2000), (fill, 1), (few, 7000)]
    got = T.summary(["one", "two"], table("t.csv", True, rows), table("f.csv", False, rows), table("w.csv", False, rows))
    assert got.splitlines()[2:] == ["| one | attn_few_kernel<float, 64> | 5.0 | 5.12 | 5.12 |",
                                    "|  | attn_join_kernel<bf16, 64> | 2.0 | 2.05 | 2.05 |",
                                    "| two | attn_few_kernel<float, 64> | 7.0 | 7.17 | 7.17 |"]
    assert T.kernel_of("_ZN3gdn12_GLOBAL__N_116attn_pair_kernelIDF16_EEvNS_8AttnArgsE") == "attn_pair_kernel<f16>"
    assert T.kernel_of("_ZN3gdn12_GLOBAL__N_118accept_walk_kernelENS_10AcceptArgsEi") == "accept_walk_kernel"
    assert T.kernel_of("gdn::(anonymous namespace)::kv_commit_kernel(gdn::AttnDims, int)") == "kv_commit_kernel"
