"""moe_sort and moe_w4a16_gemm where their launches change: tokens sorted in one
launch or two, tiles of 16, 32 and 128 rows."""
import pytest
import torch

from tests.test_gpu_moe_sorted import check_ffn, check_order, experts_of, gen, ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def nvm():
    import nvfp4_w4a16_mtp_amd as nv
    return nv


@pytest.mark.parametrize("m", [23, 24, 25, 26, 48])
@pytest.mark.parametrize("experts,k", [(2, 2), (256, 8), (1023, 16)])
def test_tokens_in_one_launch_and_two(nvm, m, experts, k):
    logits = torch.randn((m, experts), generator=gen(m))
    ws = nvm.moe_sort_workspace(m, k, experts, "cuda")
    ws.random_(0, 256)
    o = nvm.moe_sort(logits.cuda(), k, workspace=ws)
    ids, _ = ref.route(logits, k)
    assert o.topk_ids.tolist() == ids.tolist()
    check_order(o, ids, experts)
    given = nvm.moe_sort(None, topk_ids=o.topk_ids, experts=experts)
    check_order(given, ids, experts)


@pytest.mark.parametrize("per", [12, 13, 32, 33])
def test_rows_an_expert_at_which_tiles_grow(nvm, per):
    dev, vals = experts_of(nvm, 4, 96, 64, per)
    x = torch.randn((per * 2, 96), generator=gen(per)).to(torch.bfloat16).cuda()
    check_ffn(nvm, x, torch.randn((per * 2, 4), generator=gen(per + 1)), 2, dev, vals)
