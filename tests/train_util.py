"""Device tensors for the training operators' GPU tests: values rounded to
their storage, rows inside wider buffers, and bounds that count the storage
rounding (at most half a step, eps / 2 of the type)."""

import numpy as np
import torch

DT = {"f32": torch.float32, "bf16": torch.bfloat16}


def stored(a, dtype):
    """(device tensor of `a` in the storage type, the f32 values it holds)."""
    t = torch.from_numpy(np.ascontiguousarray(a, dtype=np.float32)).to(DT[dtype])
    return t.cuda(), t.float().numpy()


def strided(t, pad, offset=0):
    """The same rows inside a wider buffer of NaN, `offset` elements in."""
    rows, cols = t.shape
    buf = torch.full((rows, cols + pad), float("nan"), dtype=t.dtype, device=t.device)
    v = buf[:, offset:offset + cols]
    v.copy_(t)
    return v


def host(t):
    return t.detach().float().cpu().numpy()


def close(got, want, bound, dtype):
    """got (a tensor of the storage type) within bound + the storage rounding of want."""
    g = got.detach().double().cpu().numpy()
    half = torch.finfo(DT[dtype]).eps / 2
    tol = bound + half * (np.abs(want) + bound)
    bad = ~(np.abs(g - want) <= tol)
    assert not bad.any(), (int(bad.sum()), g[bad][:4], want[bad][:4], np.broadcast_to(tol, g.shape)[bad][:4])


def same_bits(got, want_f32, dtype):
    """got equal, bit for bit, to the f32 values rounded once to the storage type (NaN for NaN)."""
    w = torch.from_numpy(np.ascontiguousarray(want_f32, dtype=np.float32)).to(DT[dtype])
    g = got.detach().cpu().contiguous()
    view = torch.int32 if dtype == "f32" else torch.int16
    ok = (g.view(view) == w.view(view)) | (g.isnan() & w.isnan())
    assert bool(ok.all()), (int((~ok).sum()), g[~ok][:4], w[~ok][:4])


def scratch(n):
    """A poisoned workspace of exactly n bytes (16 at least)."""
    return torch.full((max(16, n),), 0xA5, dtype=torch.uint8, device="cuda")
