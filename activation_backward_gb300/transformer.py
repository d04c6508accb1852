"""Layer norm, attention's backward pass and orthogonalised updates on torch
tensors: shapes, strides and types are read from the tensors, outputs and
workspaces come from torch's allocator, and the calls go to the current stream.

PyTorch is used only for device memory and streams; every arithmetic step runs
in libcba's kernels.
"""
import torch

from . import _binding as B


def _rows(t):
    """t as [rows, cols] without a copy."""
    r = t.reshape(-1, t.shape[-1])
    if t.numel() and r.data_ptr() != t.data_ptr():
        raise ValueError("the leading axes of the tensor do not fold into one")
    if t.numel() and t.shape[-1] > 1 and r.stride(1) != 1:
        raise ValueError("the innermost axis is not contiguous")
    # (an expanded tensor's stride of 0 would read as the descriptor's "contiguous")
    if t.numel() and r.shape[0] > 1 and r.stride(0) < r.shape[1]:
        raise ValueError("rows of the tensor lie on one another (it is expanded): make it contiguous")
    return r


def _on_device_of(x, **others):
    for name, t in others.items():
        if t is not None and t.device != x.device:
            raise ValueError(f"{name} is on {t.device}, not on {x.device}")


def _workspace(nbytes, what, device):
    if nbytes == 0:
        raise B.CbaError(B.CBA_ERR_ARG, what)
    return torch.empty(nbytes, dtype=torch.uint8, device=device)


def _check_status(ws, what):
    code = B.cba_get_status(ws)
    if code != B.CBA_OK:
        raise B.CbaError(code, what)


def _norm_desc(x, gamma, beta, eps, **strides):
    for p in (gamma, beta):
        if p is not None and (p.shape != x.shape[-1:] or not p.is_contiguous()):
            raise ValueError("gamma and beta are contiguous vectors of x's last axis")
    if gamma is not None and beta is not None and gamma.dtype != beta.dtype:
        raise TypeError("gamma and beta differ in type")
    par = next((p.dtype for p in (gamma, beta) if p is not None), torch.float32)
    return B.make_layernorm_desc(x.shape[0], x.shape[1], type=B.dtype_code(x.dtype),
                                 param_type=B.dtype_code(par), eps=eps, **strides)


def _ld(t):
    return t.stride(0) if t.shape[0] > 1 else 0


def layer_norm(x, gamma=None, beta=None, eps=1e-5):
    """(y, mean, rstd) over the last axis of x; mean and rstd (fp32, one per
    row) are what the backward pass takes.  x: any row stride, but no expanded rows."""
    rows = _rows(x)
    _on_device_of(x, gamma=gamma, beta=beta)
    y = torch.empty(x.shape, dtype=x.dtype, device=x.device)
    mean, rstd = (torch.empty(rows.shape[0], dtype=torch.float32, device=x.device) for _ in range(2))
    d = _norm_desc(rows, gamma, beta, eps, ld_x=_ld(rows))
    B.cba_layernorm_forward(d, rows, gamma, beta, y, mean, rstd)
    return y, mean, rstd


def layer_norm_backward(x, dy, gamma, mean, rstd, residual=None, dgamma=None, dbeta=None):
    """(dx, dgamma, dbeta); ``residual`` (the shortcut's delta) is added to dx.
    Given dgamma and dbeta (fp32) are added to, otherwise new ones are made."""
    if dy.shape != x.shape or dy.dtype != x.dtype:
        raise ValueError("dy has another shape or type than x")
    if residual is not None and (residual.shape != x.shape or residual.dtype != x.dtype):
        raise ValueError("residual has another shape or type than x")
    if (dgamma is None) != (dbeta is None):
        raise ValueError("dgamma and dbeta come together")
    _on_device_of(x, dy=dy, gamma=gamma, mean=mean, rstd=rstd, residual=residual, dgamma=dgamma, dbeta=dbeta)
    rows, drows = _rows(x), _rows(dy)
    for t in (mean, rstd):
        if t.dtype != torch.float32 or t.numel() != rows.shape[0] or not t.is_contiguous():
            raise ValueError("mean and rstd are contiguous fp32, one element per row of x")
    rrows = None if residual is None else _rows(residual)
    dx = torch.empty(x.shape, dtype=x.dtype, device=x.device)
    add = dgamma is not None
    if not add:
        dgamma, dbeta = (torch.empty(x.shape[-1], dtype=torch.float32, device=x.device) for _ in range(2))
    for g in (dgamma, dbeta):
        if g.dtype != torch.float32 or g.shape != x.shape[-1:] or not g.is_contiguous():
            raise ValueError("dgamma and dbeta are contiguous fp32 vectors of x's last axis")
    d = _norm_desc(rows, gamma, None, 0.0, ld_x=_ld(rows), ld_dy=_ld(drows),
                   ld_residual=0 if rrows is None else _ld(rrows), accumulate=int(add))
    ws = _workspace(B.cba_layernorm_workspace_bytes(d), "cba_layernorm_workspace_bytes", x.device)
    B.cba_layernorm_backward(d, rows, drows, gamma, mean, rstd, rrows, dx, dgamma, dbeta, ws)
    return dx, dgamma, dbeta


def attention_backward(q, k, v, o, lse, dout, causal=False, scale=None, cu_q=None, cu_k=None,
                       max_q=None, max_k=None, check=False):
    """(dq, dk, dv) of softmax(scale q k^T) v.

    Dense: [batch, len, heads, dim] tensors of any strides, lse fp32 [batch,
    heads, len].  Packed: [tokens, heads, dim] with cu_q and cu_k (int32 starts
    of the sequences, one more than there are; cu_k defaults to cu_q) and lse
    [heads, tokens]; the starts run from 0 to the number of tokens (rows of tokens
    outside are not written).  max_q and max_k: upper bounds of the sequences' lengths
    (default: all tokens).  check: wait for the call and raise if one of its device
    waits ran out.  Expanded tensors, and tensors of another device, are refused."""
    outs = [torch.empty(t.shape, dtype=t.dtype, device=t.device) for t in (q, k, v)]
    _on_device_of(q, lse=lse, cu_q=cu_q, cu_k=cu_k)
    sequences = None
    if cu_q is not None:
        cu_k = cu_q if cu_k is None else cu_k
        for c in (cu_q, cu_k):
            if c.dtype != torch.int32 or not c.is_contiguous() or c.numel() != cu_q.numel():
                raise ValueError("cu_q and cu_k are contiguous int32 vectors of one length")
        sequences = cu_q.numel() - 1
    want = (*q.shape[:-3], q.shape[-2], q.shape[-3])
    if lse.dtype != torch.float32 or tuple(lse.shape) != want or not lse.is_contiguous():
        raise ValueError(f"lse is contiguous fp32 {list(want)}")
    d = B.make_attention_desc(q, k, v, o, dout, *outs, causal=causal, scale=scale,
                              sequences=sequences, max_q=max_q, max_k=max_k)
    ws = _workspace(B.cba_attention_workspace_bytes(d), "cba_attention_workspace_bytes", q.device)
    B.cba_attention_backward(d, q, k, v, o, lse, dout, cu_q, cu_k, *outs, ws)
    if check:
        _check_status(ws, "cba_attention_backward")
    return tuple(outs)


def orthogonalize(G, steps=5, coefficients=B.NEWTON_SCHULZ, eps=1e-7, scale=1.0,
                  out_dtype=torch.bfloat16, check=False):
    """The Newton-Schulz iterate of each matrix of G [..., rows, cols] (a
    convolution's dW [K, C, R, S] as dW.view(K, -1)).  check: wait for the call and
    raise if one of its device waits ran out."""
    g = G.reshape(-1, *G.shape[-2:]).contiguous()
    out = torch.empty(G.shape, dtype=out_dtype, device=G.device)
    d = B.make_orthogonalize_desc(*g.shape, in_type=B.dtype_code(G.dtype),
                                  out_type=B.dtype_code(out_dtype), steps=steps,
                                  coefficients=coefficients, eps=eps, scale=scale)
    ws = _workspace(B.cba_orthogonalize_workspace_bytes(d), "cba_orthogonalize_workspace_bytes",
                    G.device)
    B.cba_orthogonalize(d, g, out, ws)
    if check:
        _check_status(ws, "cba_orthogonalize")
    return out
