"""The decode as the first CUDA work of a thread, over a cache that no call has seen: nothing is allocated in the
thread and no other call comes before."""
import threading

import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kind", ["bf16", "split", "e4m3"])
def test_first_cuda_work_of_a_thread(kind):
    import paged_mla_decode_10_gb300 as M
    dt = torch.float8_e4m3fn if kind == "e4m3" else torch.bfloat16
    g = torch.Generator(device="cuda").manual_seed(3)
    q = torch.randn((2, 1, 16, 576), generator=g, device="cuda").to(dt)
    cache = torch.randn((12, 64, 1, 576), generator=g, device="cuda").to(dt)
    bt = torch.arange(12, dtype=torch.int32, device="cuda").view(2, 6)
    L = torch.tensor([300, 70], dtype=torch.int32, device="cuda")
    md, ns = M.mla_get_metadata(L, 16, 1, kv_dtype=dt)
    ws = torch.empty(1 << 26, dtype=torch.uint8, device="cuda")

    def decode(q, cache, **kw):
        if kind == "e4m3":
            return M.mla_decode_fwd_fp8(q, cache, bt, L, 512, md, ns, 0.04, workspace=ws, **kw)
        if kind == "bf16":
            return M.mla_decode_fwd(q, cache, bt, L, 512, md, ns, workspace=ws, **kw)
        return M.mla_decode_fwd_split(q[..., :512], q[..., 512:], cache[..., :512], cache[..., 512:], bt, L, 512, md, ns,
                                      workspace=ws, **kw)

    want = decode(q, cache)
    q2, cache2 = q.clone(), cache.clone()          # at addresses of their own
    out, lse = torch.empty_like(want[0]), torch.empty_like(want[1])
    torch.cuda.synchronize()
    failed = []

    def work():
        try:
            decode(q2, cache2, out=out, softmax_lse=lse)
        except Exception as e:
            failed.append(e)

    t = threading.Thread(target=work)
    t.start()
    t.join()
    torch.cuda.synchronize()
    assert not failed and torch.equal(out, want[0]) and torch.equal(lse, want[1]), failed
