"""Layer norm, attention, query and key norms with rotation, dropout and
orthogonalised updates on torch tensors: shapes, strides and types are read from the tensors, outputs and
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


def _sequences(q, cu_q, cu_k):
    """(cu_k, sequences) of a call; sequences is None when dense."""
    if cu_q is None:
        return cu_k, None
    cu_k = cu_q if cu_k is None else cu_k
    for c in (cu_q, cu_k):
        if c.dtype != torch.int32 or not c.is_contiguous() or c.numel() != cu_q.numel():
            raise ValueError("cu_q and cu_k are contiguous int32 vectors of one length")
    return cu_k, cu_q.numel() - 1


def attention(q, k, v, causal=False, scale=None, cu_q=None, cu_k=None, max_q=None, max_k=None, check=False):
    """(o, lse) of softmax(scale q k^T) v, what attention_backward takes.

    Tensors, sequences and bounds as of attention_backward: dense [batch, len, heads,
    dim] of any strides with lse fp32 [batch, heads, len], or packed [tokens, heads, dim]
    with cu_q and cu_k and lse [heads, tokens].  Rows that see no key get o = 0 and lse =
    -inf.  Packed tokens outside the starts are not written.  check: wait for the call
    and raise if one of its device waits ran out."""
    o = torch.empty(q.shape, dtype=q.dtype, device=q.device)
    _on_device_of(q, cu_q=cu_q, cu_k=cu_k)
    cu_k, sequences = _sequences(q, cu_q, cu_k)
    d = B.make_attention_desc(q, k, v, o, causal=causal, scale=scale, sequences=sequences, max_q=max_q,
                              max_k=max_k)
    lse = torch.empty((*q.shape[:-3], q.shape[-2], q.shape[-3]), dtype=torch.float32, device=q.device)
    ws = _workspace(B.cba_attention_forward_workspace_bytes(d), "cba_attention_forward_workspace_bytes", q.device)
    B.cba_attention_forward(d, q, k, v, cu_q, cu_k, o, lse, ws)
    if check:
        _check_status(ws, "cba_attention_forward")
    return o, lse


def _qk_params(q, k, gamma_q, gamma_k, table, pos, norm):
    """(param_type, rot_dim, positions) of a call."""
    _on_device_of(q, k=k, gamma_q=gamma_q, gamma_k=gamma_k, table=table, pos=pos)
    given = [g for g in (gamma_q, gamma_k) if g is not None]
    for g in given:
        if g.shape != q.shape[-1:] or not g.is_contiguous():
            raise ValueError("gamma_q and gamma_k are contiguous vectors of the heads' elements")
        if g.dtype != given[0].dtype:
            raise TypeError("gamma_q and gamma_k differ in type")
    if given and not norm:
        raise ValueError("gamma_q and gamma_k come with the norm")
    if table is not None and (table.dtype != torch.float32 or table.dim() != 3 or table.shape[2] != 2 or
                              not table.is_contiguous()):
        raise ValueError("table is contiguous fp32 [positions, rot_dim / 2, 2]")
    if pos is not None and (pos.dtype != torch.int32 or not pos.is_contiguous() or pos.shape != q.shape[:-2]):
        raise ValueError(f"pos is contiguous int32 {list(q.shape[:-2])}")
    par = B.dtype_code(given[0].dtype) if given else B.CBA_F32
    return (par, 0, 0) if table is None else (par, 2 * table.shape[1], table.shape[0])


def qk_norm_rope(q, k, gamma_q=None, gamma_k=None, table=None, pos=None, norm=True, interleaved=False, eps=1e-6):
    """(yq, yk): every head of q and k over its root mean square, times gamma, its first
    rot_dim elements turned by the angles of its token's position.

    q, k: [batch, len, heads, dim] or one sequence [len, heads, dim] of any strides; k may
    be None (then yk is).  table: fp32 [positions, rot_dim / 2, 2], cos and sin of
    every position's angles (None: no rotation).  pos: int32 [batch, len], the tokens'
    rows of the table (None: their index in the sequence).  interleaved: pairs (2j, 2j +
    1) instead of (j, j + rot_dim / 2).  norm=False: the rotation alone."""
    par, rot, positions = _qk_params(q, k, gamma_q, gamma_k, table, pos, norm)
    yq, yk = (None if t is None else torch.empty(t.shape, dtype=t.dtype, device=t.device) for t in (q, k))
    d = B.make_qk_norm_rope_desc(q, k, yq=yq, yk=yk, rot_dim=rot, interleaved=interleaved, positions=positions,
                                 norm=norm, eps=eps, param_type=par)
    B.cba_qk_norm_rope_forward(d, q, k, gamma_q, gamma_k, table, pos, yq, yk)
    return yq, yk


def qk_norm_rope_backward(q, k, dyq, dyk, gamma_q=None, gamma_k=None, table=None, pos=None, norm=True,
                          interleaved=False, eps=1e-6, dgamma_q=None, dgamma_k=None):
    """(dq, dk, dgamma_q, dgamma_k) from the forward's inputs and the gradients of its
    outputs.  Given dgamma_q and dgamma_k (fp32) are added to, otherwise new ones are made
    (None without the norm)."""
    par, rot, positions = _qk_params(q, k, gamma_q, gamma_k, table, pos, norm)
    if (dyq is None) != (q is None) or (dyk is None) != (k is None):
        raise ValueError("dyq comes with q, dyk with k")
    sides = [q] if k is None else [q, k]
    add = dgamma_q is not None or dgamma_k is not None
    if add and (not norm or (dgamma_q is None) or (dgamma_k is None) != (k is None)):
        raise ValueError("dgamma_q and dgamma_k come together, and with the norm")
    _on_device_of(q, dgamma_q=dgamma_q, dgamma_k=dgamma_k)
    dq, dk = (None if t is None else torch.empty(t.shape, dtype=t.dtype, device=t.device) for t in (q, k))
    if norm and not add:
        dgs = [torch.empty(q.shape[-1], dtype=torch.float32, device=q.device) for _ in sides]
        dgamma_q, dgamma_k = (dgs + [None])[:2]
    for g in (dgamma_q, dgamma_k):
        if g is not None and (g.dtype != torch.float32 or g.shape != q.shape[-1:] or not g.is_contiguous()):
            raise ValueError("dgamma_q and dgamma_k are contiguous fp32 vectors of the heads' elements")
    d = B.make_qk_norm_rope_desc(q, k, dyq=dyq, dyk=dyk, dq=dq, dk=dk, rot_dim=rot, interleaved=interleaved,
                                 positions=positions, norm=norm, eps=eps, param_type=par, accumulate=int(add))
    ws = _workspace(B.cba_qk_norm_rope_workspace_bytes(d), "cba_qk_norm_rope_workspace_bytes", q.device)
    B.cba_qk_norm_rope_backward(d, q, k, gamma_q, gamma_k, table, pos, dyq, dyk, dq, dk, dgamma_q, dgamma_k, ws)
    return dq, dk, dgamma_q, dgamma_k


def dropout(x, p, seed, offset=0, residual=None, step=None):
    """x / (1 - p) where an element's random word keeps it, 0 elsewhere, plus the residual
    (the shortcut).  The words are a function of the seed, the counter and the element's
    index: the gradient is the same call on dy without the residual.  A call uses
    (x.numel() + 3) // 4 counters from ``offset`` (plus ``step``, one int64 element on the
    device, read when the call runs) on.  x, residual: any row stride, but no expanded rows."""
    if residual is not None and (residual.shape != x.shape or residual.dtype != x.dtype):
        raise ValueError("residual has another shape or type than x")
    if step is not None and (step.dtype != torch.int64 or step.numel() != 1):
        raise ValueError("step is one int64 element")
    _on_device_of(x, residual=residual, step=step)
    rows = _rows(x)
    rrows = None if residual is None else _rows(residual)
    y = torch.empty(x.shape, dtype=x.dtype, device=x.device)
    d = B.make_dropout_desc(rows.shape[0], rows.shape[1], type=B.dtype_code(x.dtype), p=p, seed=seed, offset=offset,
                            ld_x=_ld(rows), ld_residual=0 if rrows is None else _ld(rrows))
    B.cba_dropout(d, rows, rrows, step, y)
    return y


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
    cu_k, sequences = _sequences(q, cu_q, cu_k)
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
