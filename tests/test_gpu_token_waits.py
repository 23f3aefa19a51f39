"""Expired waits of the exact token cache's attention: a hand-off that the first
block over the prefix leaves undone, with every wait limited to milliseconds."""
import pytest
import torch

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.fixture(scope="module")
def R():
    import kv_cache_vector_segmented_b200 as R
    return R


# B, H, G, P, (sequence, head) pairs that the first block has a share of: one key
# tile, several with one row tile, a pair of row tiles beside a single one
CASES = [(1, 1, 1, 50, lambda b, h: True), (2, 2, 4, 40000, lambda b, h: h == 0),
         (65, 1, 4, 20011, lambda b, h: b < 64)]


@pytest.mark.parametrize("hand_off", [1, 2])
@pytest.mark.parametrize("case", range(len(CASES)))
def test_expired_wait_poisons_its_rows_only(R, case, hand_off):
    B, H, G, P, hit = CASES[case]
    cap = 40
    g = torch.Generator().manual_seed(case)
    c = R.TokenCache.empty(B, H, G, cap, DEV)
    c.K.copy_(torch.randn(c.K.shape, generator=g))
    c.V.copy_(torch.randn(c.V.shape, generator=g))
    c.lens.copy_(torch.randint(1, cap + 1, (B, H), generator=g))
    w0 = torch.rand(B, H, cap, generator=g).to(DEV)
    prefix = tuple(torch.randn(H, P, 128, generator=g).bfloat16().to(DEV) for _ in range(2))
    q = torch.randn(B, H * G, 128, generator=g).bfloat16().to(DEV)
    ws = R.alloc_workspace(R.token_attend_workspace_bytes(c, P), DEV)

    def call(fn, *args):
        c.weight.copy_(w0)
        out, lse = fn(q, c, prefix, *args)
        status = R.read_device_status(ws)
        return out.view(B, H, G, 128), lse.view(B, H, G), c.weight.clone(), status

    def plain(q, c, prefix):
        return R.token_attend(q, c, prefix, workspace=ws)

    out, lse, weight, status = call(plain)
    assert status == 0
    # the workspace now holds a whole call's shares: none of them may be taken up again
    got = call(R.selftest_token_attend_timeout, ws, hand_off, 2_000_000)
    assert got[3] == R.STATUS_CODES["RI_ERR_TIMEOUT"]
    lost = torch.tensor([[hit(b, h) for h in range(H)] for b in range(B)], device=DEV)
    assert got[0][lost].isnan().all() and got[1][lost].isnan().all()
    assert torch.equal(got[2][lost], w0[lost])
    assert torch.equal(got[0][~lost], out[~lost]) and torch.equal(got[1][~lost], lse[~lost])
    assert torch.equal(got[2][~lost], weight[~lost])
    # the next call is right again
    again = call(plain)
    assert again[3] == 0
    for a, b in zip(again[:3], (out, lse, weight)):
        assert torch.equal(a, b)
