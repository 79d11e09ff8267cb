"""The few-token layer's slices of mlp, read off its workspace on the CPU: a share of fp32 per slot and slice."""
import pytest

import mixture_experts_ffn_group_amd as moe


def _slices(T, emb, mlp, E, k):
    run = -(-emb // 4096) * 64  # rows of emb of a router wave; four waves a workgroup
    logits = -(-(-(-emb // (4 * run)) * T * E * 8) // 256) * 256
    return (moe.workspace_bytes_few(T, emb, mlp, E, k) - logits) / (T * k * emb * 4)


# The sizes are those at which both widths were timed (bf16; the workspace fits the width that takes more).
@pytest.mark.parametrize("T,emb,mlp,E,k,width", [
    (4, 2048, 768, 128, 8, 128), (5, 2048, 768, 128, 8, 128), (6, 2048, 768, 128, 8, 64), (7, 2048, 768, 128, 8, 64),
    (8, 2048, 768, 128, 8, 64), (10, 2048, 768, 128, 8, 64), (12, 2048, 768, 128, 8, 128), (64, 2048, 768, 128, 8, 128),
    (5, 2048, 1408, 64, 6, 64), (7, 2048, 1408, 64, 6, 64), (8, 2048, 1408, 64, 6, 128), (16, 2048, 1408, 64, 6, 128),
    (10, 1024, 512, 128, 8, 128), (12, 1024, 512, 128, 8, 64), (16, 1024, 512, 128, 8, 64),
    (64, 1024, 512, 128, 8, 128),
    (2, 7168, 2048, 64, 8, 128), (3, 7168, 2048, 64, 8, 128), (8, 7168, 2048, 64, 8, 128), (4, 7168, 2048, 256, 8, 128),
    (7, 4096, 1536, 64, 4, 64), (8, 4096, 1536, 64, 4, 64), (10, 4096, 1536, 64, 4, 128), (8, 4096, 14336, 8, 2, 128),
    (10, 5120, 1024, 64, 6, 128)])
def test_slices_go_by_the_experts_that_are_expected_to_have_tokens(T, emb, mlp, E, k, width):
    assert round(_slices(T, emb, mlp, E, k), 2) == -(-mlp // width)
