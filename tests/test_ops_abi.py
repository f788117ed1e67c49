"""Refusals of the operators next to the owner step (no GPU: every case is
turned away by the host checks, on fake pointers)."""
import pytest

BF, F32 = 1, 0
A, B, C, D, WS = 0x10000000, 0x20000000, 0x30000000, 0x40000000, 0x50000000    # fake, aligned, far apart


def test_grad_clip_refusals(mfsdp):
    lib = mfsdp.raw_lib()
    wsb = lib.mfsdp_grad_clip_workspace_bytes(2)
    assert wsb > 0 and lib.mfsdp_grad_clip_workspace_bytes(-1) == 0
    assert lib.mfsdp_grad_clip_workspace_bytes(5000) > wsb

    def call(ts=((A, B, 1000, F32, F32), (C, D, 1000, BF, BF)), fn=lib.mfsdp_grad_clip, n=None, max_norm=1.0, eps=1e-6,
             out=WS + (1 << 24), ws=WS, bytes_=wsb):
        arr = (mfsdp.GradTensor * max(len(ts), 1))()
        for a, t in zip(arr, ts):
            a.src, a.dst, a.numel, a.src_dtype, a.dst_dtype = t
        return fn(arr, len(ts) if n is None else n, max_norm, eps, out, ws, bytes_, None)

    assert call(max_norm=-1.0) == call(max_norm=float("nan")) == mfsdp.ERR_INVALID_ARG
    assert call(eps=-1e-9) == call(eps=float("inf")) == call(n=-1) == mfsdp.ERR_INVALID_ARG
    assert call(out=None) == call(ws=None) == mfsdp.ERR_INVALID_ARG
    assert call(ts=((None, B, 10, F32, F32),)) == call(ts=((A, None, 10, F32, F32),)) == mfsdp.ERR_INVALID_ARG
    assert call(ts=((A, B, -1, F32, F32),)) == mfsdp.ERR_INVALID_ARG
    assert call(ts=((A, B, 10, 2, F32),)) == call(ts=((A, B, 10, F32, 7),)) == mfsdp.ERR_UNSUPPORTED_DTYPE
    assert call(ts=((A + 2, B, 10, F32, F32),)) == call(ts=((A, B + 1, 10, F32, BF),)) == mfsdp.ERR_MISALIGNED
    assert call(ws=WS + 128) == call(out=WS + (1 << 24) + 4) == mfsdp.ERR_MISALIGNED
    assert call(bytes_=wsb - 1) == mfsdp.ERR_WORKSPACE_TOO_SMALL
    assert call(ts=((A, B, 1 << 47, BF, BF),)) == mfsdp.ERR_UNSUPPORTED_SHAPE
    # destinations over each other, another source, their own source shifted or of another dtype
    assert call(ts=((A, B, 100, F32, F32), (C, B + 396, 100, F32, F32))) == mfsdp.ERR_OVERLAP
    assert call(ts=((A, B, 100, F32, F32), (B, D, 100, F32, F32))) == mfsdp.ERR_OVERLAP
    assert call(ts=((A, A + 4, 100, F32, F32),)) == call(ts=((A, A, 100, F32, BF),)) == mfsdp.ERR_OVERLAP
    # a long source before a short one still hides the destination inside it
    assert call(ts=((A, B, 1000, F32, F32), (A + 16, A + 800, 4, F32, F32))) == mfsdp.ERR_OVERLAP
    assert call(ts=((A, A, 100, F32, F32), (A, A, 100, F32, F32))) == mfsdp.ERR_OVERLAP
    assert call(out=A) == call(out=B) == call(out=WS) == call(ws=A) == mfsdp.ERR_OVERLAP
    # the norm alone looks at no destination
    assert call(fn=lib.mfsdp_grad_norm, ts=((A, None, 10, F32, 9),), ws=WS + 8) == mfsdp.ERR_MISALIGNED


def test_sort_and_embedding_refusals(mfsdp):
    lib = mfsdp.raw_lib()
    assert lib.mfsdp_sort_ids_workspace_bytes(-1, 5) == lib.mfsdp_sort_ids_workspace_bytes(5, 0) == 0
    sb = lib.mfsdp_sort_ids_workspace_bytes(1000, 50)

    def sort(ids=A, it=mfsdp.ID_I64, n=1000, keys=50, order=B, starts=C, ws=WS, bytes_=sb):
        return lib.mfsdp_sort_ids(ids, it, n, keys, order, starts, ws, bytes_, None)
    assert sort(it=2) == mfsdp.ERR_UNSUPPORTED_DTYPE
    assert sort(n=-1) == sort(keys=0) == sort(ids=None) == sort(order=None) == sort(starts=None) == sort(ws=None) \
        == mfsdp.ERR_INVALID_ARG
    assert sort(n=1 << 31) == sort(keys=(1 << 31) - 1) == mfsdp.ERR_UNSUPPORTED_SHAPE
    assert sort(ids=A + 4) == sort(order=B + 2) == sort(ws=WS + 16) == mfsdp.ERR_MISALIGNED
    assert sort(bytes_=sb - 1) == mfsdp.ERR_WORKSPACE_TOO_SMALL
    assert sort(order=A) == sort(starts=B + 400) == sort(ws=A) == mfsdp.ERR_OVERLAP

    def lookup(w=A, wdt=F32, vocab=100, dim=64, w_ld=64, ids=B, it=mfsdp.ID_I32, n=10, scale=1.0, out=C, odt=BF,
               o_ld=64):
        return lib.mfsdp_embedding_lookup(w, wdt, vocab, dim, w_ld, ids, it, n, scale, out, odt, o_ld, None)
    assert lookup(n=0, ids=None, out=None, w=None) == mfsdp.OK
    assert lookup(wdt=3) == lookup(odt=-1) == lookup(it=9) == mfsdp.ERR_UNSUPPORTED_DTYPE
    assert lookup(dim=0) == lookup(vocab=0) == lookup(n=-1) == lookup(scale=float("nan")) == lookup(w=None) \
        == lookup(out=None) == lookup(ids=None) == mfsdp.ERR_INVALID_ARG
    assert lookup(w_ld=63) == lookup(o_ld=63) == lookup(dim=1 << 25, w_ld=1 << 25, o_ld=1 << 25) \
        == mfsdp.ERR_UNSUPPORTED_SHAPE
    assert lookup(w=A + 8) == lookup(out=C + 2) == lookup(ids=B + 2) == mfsdp.ERR_MISALIGNED
    assert lookup(out=A) == lookup(out=A + 100 * 256 - 16) == lookup(ids=C) == mfsdp.ERR_OVERLAP

    assert lib.mfsdp_embedding_grad_workspace_bytes(10, 0, 64) == 0
    gb = lib.mfsdp_embedding_grad_workspace_bytes(10, 100, 64)

    def grad(do=A, ddt=BF, d_ld=64, ids=B, it=mfsdp.ID_I32, n=10, scale=1.0, g=C, gdt=F32, vocab=100, dim=64, g_ld=64,
             acc=0, ws=WS, bytes_=gb):
        return lib.mfsdp_embedding_grad(do, ddt, d_ld, ids, it, n, scale, g, gdt, vocab, dim, g_ld, acc, ws, bytes_,
                                        None)
    assert grad(n=0, do=None, ids=None, acc=1) == mfsdp.OK
    assert grad(ddt=4) == grad(gdt=4) == grad(it=4) == mfsdp.ERR_UNSUPPORTED_DTYPE
    assert grad(acc=2) == grad(do=None) == grad(g=None) == grad(ids=None) == grad(ws=None) \
        == grad(scale=float("inf")) == mfsdp.ERR_INVALID_ARG
    assert grad(d_ld=8) == grad(g_ld=63) == mfsdp.ERR_UNSUPPORTED_SHAPE
    assert grad(do=A + 2) == grad(g=C + 4) == grad(ws=WS + 64) == mfsdp.ERR_MISALIGNED
    assert grad(bytes_=gb - 1) == mfsdp.ERR_WORKSPACE_TOO_SMALL
    assert grad(g=A) == grad(ws=C) == grad(ws=B) == mfsdp.ERR_OVERLAP


def test_expert_refusals(mfsdp):
    lib = mfsdp.raw_lib()
    E, R, K, N = 4, 64, 96, 100
    q = lib.mfsdp_expert_workspace_bytes
    assert q(0, N, R, K, R * K, R, K) == q(E, N, R, K, R * K - 1, R, K) == q(E, N, R, K, R * K, R - 1, K) == 0
    assert q(2000, N, R, K, R * K, R, K) == q(E, -1, R, K, R * K, R, K) == 0
    wsb = q(E, N, R, K, R * K, R, K)

    def mm(x=A, x_ld=K, w=B, ws_=R * K, dt=BF, st=C, e=E, n=N, r=R, k=K, ig=0, y=D, ydt=BF, y_ld=R, ws=WS, bytes_=wsb):
        return lib.mfsdp_expert_matmul(x, x_ld, w, ws_, dt, st, e, n, r, k, ig, y, ydt, y_ld, ws, bytes_, None)
    assert mm(n=0, x=None, y=None, st=None) == mfsdp.OK
    assert mm(dt=F32) == mm(ydt=5) == mfsdp.ERR_UNSUPPORTED_DTYPE
    assert mm(e=0) == mm(n=-1) == mm(r=0) == mm(k=0) == mm(ig=2) == mm(x=None) == mm(w=None) == mm(y=None) \
        == mm(st=None) == mm(ws=None) == mfsdp.ERR_INVALID_ARG
    assert mm(e=1025) == mm(x_ld=K - 1) == mm(y_ld=R - 1) == mm(ws_=R * K - 1) == mm(n=1 << 31) \
        == mm(ig=1) == mfsdp.ERR_UNSUPPORTED_SHAPE          # input_grad: y is cols wide
    assert mm(x=A + 2) == mm(w=B + 8) == mm(y=D + 4) == mm(st=C + 1) == mm(ws=WS + 4) == mfsdp.ERR_MISALIGNED
    assert mm(bytes_=wsb - 1) == mfsdp.ERR_WORKSPACE_TOO_SMALL
    assert mm(y=A) == mm(y=B + 16) == mm(ws=A) == mm(ws=D) == mm(y=C) == mfsdp.ERR_OVERLAP

    def wg(dy=A, dy_ld=R, x=B, x_ld=K, dt=BF, st=C, e=E, n=N, r=R, k=K, dw=D, ddt=F32, dst=R * K, acc=0, ws=WS,
           bytes_=wsb):
        return lib.mfsdp_expert_weight_grad(dy, dy_ld, x, x_ld, dt, st, e, n, r, k, dw, ddt, dst, acc, ws, bytes_,
                                            None)
    assert wg(n=0, acc=1, dw=None) == mfsdp.OK
    assert wg(dt=F32) == wg(ddt=2) == mfsdp.ERR_UNSUPPORTED_DTYPE
    assert wg(acc=-1) == wg(dw=None) == wg(dy=None) == wg(x=None) == wg(ws=None) == mfsdp.ERR_INVALID_ARG
    assert wg(dy_ld=R - 1) == wg(x_ld=1) == wg(dst=R * K - 8) == mfsdp.ERR_UNSUPPORTED_SHAPE
    assert wg(dw=D + 8) == wg(dy=A + 4) == mfsdp.ERR_MISALIGNED
    assert wg(bytes_=0) == mfsdp.ERR_WORKSPACE_TOO_SMALL
    assert wg(dw=A) == wg(dw=B) == wg(ws=D) == mfsdp.ERR_OVERLAP


def test_binding_refuses_host_and_strided_tensors(mfsdp):
    import torch
    t = torch.zeros(4, 4)
    with pytest.raises(ValueError, match="CUDA"):
        mfsdp.grad_set([t])
    with pytest.raises(ValueError, match="CUDA"):
        mfsdp.embedding_lookup(t, torch.zeros(4, dtype=torch.int64), t)
    with pytest.raises(ValueError, match="CUDA"):
        mfsdp.sort_ids(torch.zeros(4, dtype=torch.int64), 4, t, t, None)
    with pytest.raises(ValueError, match="CUDA"):
        mfsdp.expert_matmul(t, t[None], t, t, None)
