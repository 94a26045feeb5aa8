"""The head's cross entropy and the clipping of gradients where something goes wrong or
stands close: waits that run out, guards around outputs and workspaces, the checked
build."""
import time

import pytest
import torch

import dsmem_thread_block_gb300 as credit
from dsmem_thread_block_gb300 import _credit as C
from test_gpu_linear_ce import make

pytestmark = pytest.mark.gpu


def test_a_tile_that_gives_up_waits_for_its_copies_and_no_longer():
    # Two tiles, each with one wait that runs out after a second.  The copies that were
    # issued are there long before, so waiting for them takes no time: a second limit
    # spent on a stage whose other operand never comes would make four seconds.
    dev = torch.cuda.current_device()
    h, w, target = make(300, 64, 500, torch.bfloat16)
    want = credit.linear_cross_entropy_forward(h, w, target)
    assert C.credit_get_device_error(dev) == C.OK
    t0 = time.perf_counter()
    assert C.credit_selftest_tile_timeout(dev) == C.ERR_DEVICE_TIMEOUT
    took = time.perf_counter() - t0
    assert 2.0 <= took < 3.5, took
    assert C.credit_get_device_error(dev) == C.OK
    got = credit.linear_cross_entropy_forward(h, w, target)
    assert all(torch.equal(a, b) for a, b in zip(got, want))


# few tokens (whole lines and not), whole and split products and logits, several pieces,
# tiles of each shape, ragged in every direction
SHAPES = [(1, 72, 300), (1, 71, 301), (4, 65, 1000), (8, 264, 1003), (13, 264, 64007), (20, 5000, 333),
          (33, 100, 257), (64, 4104, 300), (130, 264, 700), (300, 1001, 5003), (333, 129, 20011),
          (3000, 40, 100), (8192, 40, 20000)]


def cross_entropy(tokens, hidden, vocab, dtype, precise):
    h, w, target = make(tokens, hidden, vocab, dtype, seed=tokens)
    loss, lse = credit.linear_cross_entropy_forward(h, w, target)
    grads = credit.linear_cross_entropy_backward(loss, h, w, target, lse, dlse=0.1 * lse, precise=precise)
    return (loss, lse) + tuple(grads)


def gradients(seed=0):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    out = []
    for i, n in enumerate([1, 7, 0, 8192, 8193, 100001, 33, 64, 300000, 5]):
        room = torch.randn(n + 3, generator=g, device="cuda").to(torch.bfloat16 if i % 3 else torch.float32)
        out.append(room[i % 4 if i % 4 < 3 else 1:][:n])
    return out


@pytest.mark.parametrize("precise", [False, True])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("tokens,hidden,vocab", SHAPES)
def test_the_checked_build_finds_no_index_outside(tokens, hidden, vocab, dtype, precise):
    want = cross_entropy(tokens, hidden, vocab, dtype, precise)
    with C.use_checked_build():
        got = cross_entropy(tokens, hidden, vocab, dtype, precise)
        assert C.credit_get_device_error(torch.cuda.current_device()) == C.OK
    assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("copies", [1, 8, 120])
def test_the_checked_build_clips_every_chunk(copies):
    grads = gradients() * copies
    outs = [torch.zeros_like(t) for t in grads]
    want = credit.clip_gradients(grads, 0.5, out=outs), [t.clone() for t in outs]
    with C.use_checked_build():
        got = credit.clip_gradients(grads, 0.5, out=outs)
        assert torch.equal(credit.gradient_norm(grads), got)
        assert C.credit_get_device_error(torch.cuda.current_device()) == C.OK
    assert torch.equal(got, want[0]) and all(torch.equal(a, b) for a, b in zip(outs, want[1]))


def guarded(nbytes, shift=0):
    """`nbytes` between guards of 256 bytes, and a check that these are as they were."""
    whole = torch.full((nbytes + 512 + shift,), 0xA5, dtype=torch.uint8, device="cuda")

    def untouched():
        assert bool((whole[:256 + shift] == 0xA5).all()) and bool((whole[256 + shift + nbytes:] == 0xA5).all())

    return whole[256 + shift:256 + shift + nbytes], untouched


@pytest.mark.parametrize("precise", [False, True])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("tokens,hidden,vocab", SHAPES)
def test_nothing_beside_outputs_and_a_workspace_of_the_stated_size_is_written(tokens, hidden, vocab, dtype,
                                                                               precise):
    h, w, target = make(tokens, hidden, vocab, dtype, seed=tokens)
    code = C.BF16 if dtype == torch.bfloat16 else C.F32
    es = h.element_size()
    room, checks = [], []
    for what in (0, 2 if precise else 1):
        n = C.credit_linear_ce_workspace(what, h.data_ptr(), w.data_ptr(), tokens, hidden, vocab, code,
                                         h.device.index)
        ws, check = guarded(n)
        room.append(ws)
        checks.append(check)
    loss, lse = credit.linear_cross_entropy_forward(h, w, target, workspace=room[0])
    checks[0]()
    want = credit.linear_cross_entropy_backward(loss, h, w, target, lse, precise=precise)
    for shift in (0, es):  # rows that are whole 16-byte lines where they can be, and not
        dh, check_h = guarded(h.numel() * es, shift)
        dw, check_w = guarded(w.numel() * es, shift)
        dh, dw = dh.view(dtype).view(h.shape), dw.view(dtype).view(w.shape)
        credit.linear_cross_entropy_backward(loss, h, w, target, lse, dhidden=dh, dweight=dw, workspace=room[1],
                                             precise=precise)
        for check in checks + [check_h, check_w]:
            check()
        if shift == 0:
            assert torch.equal(dh, want[0]) and torch.equal(dw, want[1])
        dh, check_h = guarded(h.numel() * es, shift)
        dw, check_w = guarded(w.numel() * es, shift)
        credit.linear_cross_entropy_backward(loss, h, w, target, lse, need_dweight=False, workspace=room[1],
                                             dhidden=dh.view(dtype).view(h.shape), precise=precise)
        credit.linear_cross_entropy_backward(loss, h, w, target, lse, need_dhidden=False, workspace=room[1],
                                             dweight=dw.view(dtype).view(w.shape), precise=precise)
        for check in checks + [check_h, check_w]:
            check()


def test_clipping_writes_nothing_beside_its_tensors():
    grads = gradients(3)
    n = C.credit_grad_workspace(C.tensors([(t.data_ptr(), 0, t.numel(), C.F32 if t.dtype == torch.float32 else C.BF16)
                                           for t in grads]), grads[0].device.index)
    ws, check = guarded(n)
    for shift in (0, 4, 12):
        outs, checks = [], [check]
        for t in grads:
            o, c = guarded(t.numel() * t.element_size(), shift)
            outs.append(o.view(t.dtype))
            checks.append(c)
        norm = credit.clip_gradients(grads, 1.0, out=outs, workspace=ws)
        factor = 1.0 / (float(norm) + 1e-6)
        for c in checks:
            c()
        for t, o in zip(grads, outs):
            assert float((o.double() - t.double() * factor).abs().max() if t.numel() else 0) <= 2.0 ** -8 * 6 * factor


def forward_workspace(tokens, hidden, vocab, code):
    return C.credit_linear_ce_workspace(0, 1 << 32, 2 << 32, tokens, hidden, vocab, code,
                                        torch.cuda.current_device())


def test_a_losss_workspace_is_bounded():
    mib = 1 << 20
    for tokens in (4096, 16384, 65536, 1 << 20, 10 ** 7):
        for vocab in (4096, 32000, 131072, 262144):
            if tokens * vocab > 1 << 40:
                continue
            # (bf16 at whole lines: nothing is packed; 4 bytes a token for its target's logit)
            assert forward_workspace(tokens, 64, vocab, C.BF16) <= 256 * mib + 4 * min(tokens, 1 << 19) + 512
            # fp32: and both operands in three terms
            packed = 6 * 64 * (tokens + vocab)
            assert forward_workspace(tokens, 64, vocab, C.F32) <= 256 * mib + packed + 4 * min(tokens, 1 << 19) + 1024


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("hidden", [24, 65])
def test_a_loss_of_several_pieces_of_tokens(hidden, dtype):
    # 131072 words leave 16 KiB a token: pieces of 16384 tokens at most, here 13824 and less
    tokens, vocab = 41001, 131072
    h, w, target = make(tokens, hidden, vocab, dtype, seed=5)
    loss, lse = credit.linear_cross_entropy_forward(h, w, target)
    for lo, hi in ((0, 13824), (13824, 27648), (27648, tokens)):
        part = credit.linear_cross_entropy_forward(h[lo:hi].clone(), w, target[lo:hi])
        assert torch.equal(loss[lo:hi], part[0]) and torch.equal(lse[lo:hi], part[1])
    with C.use_checked_build():
        again = credit.linear_cross_entropy_forward(h, w, target)
        assert C.credit_get_device_error(torch.cuda.current_device()) == C.OK
    assert torch.equal(again[0], loss) and torch.equal(again[1], lse)
    n = forward_workspace(tokens, hidden, vocab, C.BF16 if dtype == torch.bfloat16 else C.F32)
    ws, check = guarded(n)
    again = credit.linear_cross_entropy_forward(h, w, target, workspace=ws)
    check()
    assert torch.equal(again[0], loss) and torch.equal(again[1], lse)
