"""The timing tool: names of kernels with switches among their template arguments."""

from gated_deltanet_speculative_amd import round_times as T


def test_names_of_kernels_with_switches():
    assert T.kernel_of("_ZN3gdn12_GLOBAL__N_116attn_pair_kernelIDF16bLb1EEEvNS_8AttnArgsENS_8AttnPlanE") == "attn_pair_kernel<bf16, true>"
    assert T.kernel_of("_ZN3gdn12_GLOBAL__N_116attn_rows_kernelIDF16_Li128ELi64ELb0EEEvNS_8AttnArgsENS_8AttnPlanE") == \
        "attn_rows_kernel<f16, 128, 64, false>"
    assert T.kernel_of("void gdn::(anonymous namespace)::attn_few_kernel<float, 64, true>(gdn::AttnArgs, gdn::AttnPlan)") == \
        "attn_few_kernel<float, 64, true>"
    assert T.kernel_of("void gdn::(anonymous namespace)::kv_commit_kernel<0>(gdn::AttnDims, int)") == "kv_commit_kernel<0>"
