"""What a policy over token sequences has besides attention and sampling: checks and
marshalling for librlscan's gated recurrence, normalised and rotated heads, and rows of a table
by token (declared in include/rlscan.h).

Value tensors are float32, bfloat16 or float16, all of one dtype; states, rates, marks and the
heads' weights are float32.  Per-step tensors may be strided (time-major, slices of a fused
projection) as long as their last dimension is contiguous.  Scratch memory and outputs that are
not given are allocated on the call's stream.  The functions are not differentiated by
autograd: each has its backward as a function of its own.
"""
from __future__ import annotations

import ctypes

from . import policy as _p
from .policy import (_call, _flags, _on, _on_gpu, _plain, _ptr, _raw_stream, _row_stride, _strided, _values,
                     _workspace)

_N = _p._HEADS_BYTES
MARK_STEPS = 16  # RLSCAN_MARK_STEPS


_TYPES = {n: ctypes.c_int64 * (4 * n) for n in (4, 6, 7)}  # n rlscan_heads in a row


def _rows(tensors, time_major=False):
    """(array to keep alive, addresses) of [E, T, D] tensors as rlscan_heads."""
    v = []
    for x in tensors:
        s0, s1, _ = x.stride()
        v += (x.data_ptr(), s1, s0, 0) if time_major else (x.data_ptr(), s0, s1, 0)
    a = _TYPES[len(tensors)](*v)
    h = ctypes.addressof(a)
    return a, range(h, h + len(tensors) * _N, _N)


def _empty_like(x):
    """Memory for an output that takes x's place: of its shape, contiguous."""
    return _p.torch.empty_like(x) if x.is_contiguous() else _p.torch.empty(x.shape, dtype=x.dtype, device=x.device)


def _out(x, name, like):
    return _empty_like(like) if x is None else _strided(x, name, like.shape, like.dtype, like.device)


def _recurrence_inputs(x, input_gate, decay_gate, rate, done, time_major):
    _values(x, "x", 3)
    dev, dt = _on_gpu(x, "x"), x.dtype
    n0, n1, D = x.shape
    E, T = (n1, n0) if time_major else (n0, n1)
    _strided(x, "x", x.shape, dt, dev)
    _strided(input_gate, "input_gate", x.shape, dt, dev)
    _strided(decay_gate, "decay_gate", x.shape, dt, dev)
    if not isinstance(rate, _p.torch.Tensor):
        raise TypeError("rate must be a torch.Tensor")
    _plain(rate, "rate", (D,), _p.torch.float32, dev)
    return dev, dt, E, T, D, _flags(done, "done", (n0, n1), dev)


def gated_recurrence(x, input_gate, decay_gate, rate, done=None, init_state=None, *, time_major=False,
                     with_state=False, with_marks=False, reset=None, out=None, final_state=None, marks=None, stream=None):
    """A gated memory of one number a channel, over whole rows.

    Per row and channel s_t = rate sigmoid(decay_gate_t), a_t = exp(-s_t) and
    h_t = a_t h_{t-1} + sqrt(1 - a_t^2) sigmoid(input_gate_t) x_t; the step after one flagged in
    ``done`` has a_t = 0, whatever the state was: inf and NaN stay within their episode, and an
    infinite state stays infinite as long as it lasts.

    x, input_gate, decay_gate [E, T, D] (``time_major``: [T, E, D]); rate [D] float32, not
    negative; done [E, T] (or [T, E]); init_state [E, D] float32; reset [E]: rows whose step before the first
    ended an episode (the last column of the window before's done).  Returns out, h in x's dtype, followed
    by final_state [E, D] with ``with_state`` or ``final_state`` (what the next window takes as
    init_state) and by marks [E, ceil(T / 16), D] float32 with ``with_marks`` or ``marks``
    (states on the way, which the backward call takes)."""
    dev, dt, E, T, D, done = _recurrence_inputs(x, input_gate, decay_gate, rate, done, time_major)
    torch = _p.torch
    _plain(init_state, "init_state", (E, D), torch.float32, dev)
    reset = _flags(reset, "reset", (E,), dev)
    fmt = _p._DTYPES[dt]
    with _on(stream, dev):
        out = _out(out, "out", x)
        if final_state is not None:
            _plain(final_state, "final_state", (E, D), torch.float32, dev)
        elif with_state:
            final_state = torch.empty((E, D), dtype=torch.float32, device=dev)
        shape = (E, -(-T // MARK_STEPS), D)
        if marks is not None:
            _plain(marks, "marks", shape, torch.float32, dev)
        elif with_marks:
            marks = torch.empty(shape, dtype=torch.float32, device=dev)
        ws, need = _workspace("rlscan_gated_recurrence_workspace", dev, fmt, E, T, D, 0)
        keep, h = _rows((x, input_gate, decay_gate, out), time_major)
        _call("rlscan_gated_recurrence", fmt, 1 if time_major else 0, h[0], h[1], h[2], rate.data_ptr(), _ptr(done),
              _ptr(reset), _ptr(init_state), h[3], _ptr(final_state), _ptr(marks), _ptr(ws), need, E, T, D,
              _raw_stream(stream, dev))
    outs = (out,) + tuple(t for t in (final_state, marks) if t is not None)
    return outs if len(outs) > 1 else out


def gated_recurrence_backward(d_out, x, input_gate, decay_gate, rate, marks, done=None, d_final_state=None, *,
                              time_major=False, reset=None, dx=None, d_input_gate=None, d_decay_gate=None, d_rate=None,
                              d_init_state=None, stream=None):
    """Gradients of ``gated_recurrence``: (dx, d_input_gate, d_decay_gate, d_rate, d_init_state).

    d_out like the output; marks are the forward call's, the other inputs as in it;
    d_final_state [E, D], if the final state was used."""
    dev, dt, E, T, D, done = _recurrence_inputs(x, input_gate, decay_gate, rate, done, time_major)
    torch = _p.torch
    _strided(d_out, "d_out", x.shape, dt, dev)
    if not isinstance(marks, torch.Tensor):
        raise TypeError("marks must be a torch.Tensor")
    _plain(marks, "marks", (E, -(-T // MARK_STEPS), D), torch.float32, dev)
    _plain(d_final_state, "d_final_state", (E, D), torch.float32, dev)
    reset = _flags(reset, "reset", (E,), dev)
    fmt = _p._DTYPES[dt]
    with _on(stream, dev):
        dx, di, dd = _out(dx, "dx", x), _out(d_input_gate, "d_input_gate", x), _out(d_decay_gate, "d_decay_gate", x)
        dr = torch.empty_like(rate) if d_rate is None else _plain(d_rate, "d_rate", (D,), torch.float32, dev)
        dh = d_init_state
        if dh is None:
            dh = torch.empty((E, D), dtype=torch.float32, device=dev)
        else:
            _plain(dh, "d_init_state", (E, D), torch.float32, dev)
        ws, need = _workspace("rlscan_gated_recurrence_workspace", dev, fmt, E, T, D, 1)
        keep, h = _rows((d_out, x, input_gate, decay_gate, dx, di, dd), time_major)
        _call("rlscan_gated_recurrence_backward", fmt, 1 if time_major else 0, *h[:4], rate.data_ptr(),
              marks.data_ptr(), _ptr(done), _ptr(reset), _ptr(d_final_state), *h[4:], dr.data_ptr(), dh.data_ptr(), _ptr(ws), need,
              E, T, D, _raw_stream(stream, dev))
    return dx, di, dd, dr, dh


def gated_recurrence_step(x, input_gate, decay_gate, rate, state, reset=None, slots=None, *, out=None, stream=None):
    """One step of ``gated_recurrence`` for E rows; ``state`` is updated in place.

    x, input_gate, decay_gate [E, D]; rate [D] float32; state [S, D] float32; reset [E]: rows
    that start a new episode (their state is dropped unread); slots [E] int32: row e's
    state is state[slots[e]] (state[e] if not given).  A row whose slot is outside [0, S)
    gets zeros and changes nothing; two rows of a call must not share a slot.  Returns
    out [E, D]."""
    _values(x, "x", 2)
    dev, dt = _on_gpu(x, "x"), x.dtype
    torch = _p.torch
    shape = x.shape
    E, D = shape
    _strided(x, "x", shape, dt, dev)
    _strided(input_gate, "input_gate", shape, dt, dev)
    _strided(decay_gate, "decay_gate", shape, dt, dev)
    if not isinstance(rate, torch.Tensor):
        raise TypeError("rate must be a torch.Tensor")
    _plain(rate, "rate", (D,), torch.float32, dev)
    if not isinstance(state, torch.Tensor) or state.dim() != 2:
        raise ValueError("state must be a [S, D] tensor")
    S = state.shape[0]
    _plain(state, "state", (S, D), torch.float32, dev)
    reset = _flags(reset, "reset", (E,), dev)
    _plain(slots, "slots", (E,), torch.int32, dev)
    if slots is None and S < E:
        raise ValueError("state has %d slots for %d rows" % (S, E))
    with _on(stream, dev):
        out = _out(out, "out", x)
        keep = _TYPES[4](x.data_ptr(), x.stride(0), 0, 0, input_gate.data_ptr(), input_gate.stride(0), 0, 0,
                         decay_gate.data_ptr(), decay_gate.stride(0), 0, 0, out.data_ptr(), out.stride(0), 0, 0)
        h = ctypes.addressof(keep)
        _call("rlscan_gated_recurrence_step", _p._DTYPES[dt], h, h + _N, h + 2 * _N, rate.data_ptr(), _ptr(reset),
              _ptr(slots), state.data_ptr(), h + 3 * _N, E, S, D, _raw_stream(stream, dev))
    return out


def _head_rows(tensors, time_major):
    """(array to keep alive, addresses) of the [E, T, H, D] or [E, H, D] tensors as rlscan_heads."""
    v = []
    for x in tensors:
        s = x.stride()
        if len(s) == 3:
            v += (x.data_ptr(), s[0], 0, s[1])
        else:
            v += (x.data_ptr(), s[1], s[0], s[2]) if time_major else (x.data_ptr(), s[0], s[1], s[2])
    a = _TYPES[len(tensors)](*v)
    h = ctypes.addressof(a)
    return a, range(h, h + len(tensors) * _N, _N)


def _head_inputs(q, k, q_weight, k_weight, positions, rotate, time_major):
    if _p.torch is None:
        _p._import_torch()
    torch = _p.torch
    if not isinstance(q, torch.Tensor):
        raise TypeError("q must be a torch.Tensor")
    if q.dim() not in (3, 4):
        raise ValueError("q must be [E, T, H, D] or, for one step, [E, H, D], got shape %s" % (tuple(q.shape),))
    _values(q, "q", q.dim())
    _values(k, "k", q.dim())
    dev, dt = _on_gpu(q, "q"), q.dtype
    shape = tuple(q.shape)
    if len(shape) == 3:
        E, H, D = shape
        T = 1
    else:
        E, T, H, D = shape
        if time_major:
            E, T = T, E
    lead, Hk = shape[:-2], k.shape[-2]
    _strided(q, "q", shape, dt, dev)
    _strided(k, "k", lead + (Hk, D), dt, dev)
    _plain(q_weight, "q_weight", (D,), torch.float32, dev)
    _plain(k_weight, "k_weight", (D,), torch.float32, dev)
    _plain(positions, "positions", lead, torch.int32, dev)
    if rotate is None:
        rotate = 0 if positions is None else D
    rotate = int(rotate)
    if rotate < 0 or rotate > D or rotate % 2:
        raise ValueError("rotate must be even and in [0, %d], got %d" % (D, rotate))
    if rotate and positions is None:
        raise ValueError("positions must be given to rotate by them")
    return dev, dt, E, T, H, Hk, D, rotate


def norm_rotate_heads(q, k, q_weight=None, k_weight=None, positions=None, *, rotate=None, base=10000.0,
                      interleaved=False, eps=1e-6, time_major=False, q_out=None, k_out=None, stream=None):
    """Queries and keys of attention, each head normalised and rotated by its position.

    Every head x becomes w x / sqrt(mean(x^2) + eps), and the pairs of its first ``rotate``
    elements (all of them if not given) are turned by positions[e, t] base^(-2j / rotate):
    pair j is (j, j + rotate / 2), or (2j, 2j + 1) if ``interleaved``.

    q [E, T, H, D], k [E, T, Hk, D] (``time_major``: [T, E, ...]; one step: [E, H, D]), D up to
    256; q_weight, k_weight [D] float32 (None: ones); positions [E, T] (one step: [E]) int32,
    None for normalising alone.  Returns (q_out, k_out) of their shapes and dtype."""
    dev, dt, E, T, H, Hk, D, rotate = _head_inputs(q, k, q_weight, k_weight, positions, rotate, time_major)
    with _on(stream, dev):
        q_out, k_out = _out(q_out, "q_out", q), _out(k_out, "k_out", k)
        keep, h = _head_rows((q, k, q_out, k_out), time_major)
        _call("rlscan_norm_rotate_heads", _p._DTYPES[dt], 1 if time_major and q.dim() == 4 else 0, h[0], h[1],
              _ptr(q_weight), _ptr(k_weight), _ptr(positions), h[2], h[3], E, T, H, Hk, D, rotate, float(base),
              bool(interleaved), float(eps), _raw_stream(stream, dev))
    return q_out, k_out


def norm_rotate_heads_backward(d_q_out, d_k_out, q, k, q_weight=None, k_weight=None, positions=None, *, rotate=None,
                               base=10000.0, interleaved=False, eps=1e-6, time_major=False, dq=None, dk=None,
                               d_q_weight=None, d_k_weight=None, stream=None):
    """Gradients of ``norm_rotate_heads``: (dq, dk, d_q_weight, d_k_weight).

    d_q_out and d_k_out like the outputs, the other arguments as in the forward call.  The
    gradient of a weight that is None is None, unless its buffer is given."""
    dev, dt, E, T, H, Hk, D, rotate = _head_inputs(q, k, q_weight, k_weight, positions, rotate, time_major)
    torch = _p.torch
    _strided(d_q_out, "d_q_out", q.shape, dt, dev)
    _strided(d_k_out, "d_k_out", k.shape, dt, dev)
    with _on(stream, dev):
        dq, dk = _out(dq, "dq", q), _out(dk, "dk", k)
        _plain(d_q_weight, "d_q_weight", (D,), torch.float32, dev)
        _plain(d_k_weight, "d_k_weight", (D,), torch.float32, dev)
        if d_q_weight is None and q_weight is not None:
            d_q_weight = torch.empty_like(q_weight)
        if d_k_weight is None and k_weight is not None:
            d_k_weight = torch.empty_like(k_weight)
        ws, need = _workspace("rlscan_norm_rotate_heads_workspace", dev, E, T, H, Hk, D)
        keep, h = _head_rows((d_q_out, d_k_out, q, k, dq, dk), time_major)
        _call("rlscan_norm_rotate_heads_backward", _p._DTYPES[dt], 1 if time_major and q.dim() == 4 else 0, *h[:4],
              _ptr(q_weight), _ptr(k_weight), _ptr(positions), h[4], h[5], _ptr(d_q_weight), _ptr(d_k_weight), _ptr(ws),
              need, E, T, H, Hk, D, rotate, float(base), bool(interleaved), float(eps), _raw_stream(stream, dev))
    return dq, dk, d_q_weight, d_k_weight


def _table_rows(x, name):
    """Elements between the rows of a [..., D] tensor that may have none."""
    return _row_stride(x, name) if x.numel() else x.shape[-1]


def embed_tokens(table, tokens, *, scale=1.0, out=None, stream=None):
    """Rows of a table by token, times a scale: out[...] = scale * table[tokens[...]].

    table [N, D], rows at one distance; tokens [...] int64, as ``sample_actions`` gives them:
    one outside [0, N), as for a padded step, gives zeros.  Returns out [..., D] in the
    table's dtype."""
    _values(table, "table", 2)
    dev, dt = _on_gpu(table, "table"), table.dtype
    torch = _p.torch
    N, D = table.shape
    _strided(table, "table", table.shape, dt, dev)
    if not isinstance(tokens, torch.Tensor):
        raise TypeError("tokens must be a torch.Tensor")
    _plain(tokens, "tokens", tokens.shape, torch.int64, dev)
    shape = tuple(tokens.shape) + (D,)
    with _on(stream, dev):
        out = torch.empty(shape, dtype=dt, device=dev) if out is None else _strided(out, "out", shape, dt, dev)
        _call("rlscan_embed_tokens", _p._DTYPES[dt], table.data_ptr(), _table_rows(table, "table"), tokens.data_ptr(),
              out.data_ptr(), _table_rows(out, "out"), tokens.numel(), N, D, float(scale), _raw_stream(stream, dev))
    return out


def embed_tokens_backward(d_out, tokens, N, *, scale=1.0, d_table=None, stream=None):
    """Gradient of the table of ``embed_tokens``: [N, D] in d_out's dtype.

    Row n is scale times the sum of d_out [..., D] over the tokens that are n, in float32 and
    in a fixed order: the same from run to run.  Rows without a token are zero.  An expanded
    d_out (rows that are one row) is refused: pass it as ``d_out.contiguous()``."""
    if _p.torch is None:
        _p._import_torch()
    torch = _p.torch
    if not isinstance(d_out, torch.Tensor):
        raise TypeError("d_out must be a torch.Tensor")
    _values(d_out, "d_out", d_out.dim())
    dev, dt = _on_gpu(d_out, "d_out"), d_out.dtype
    if d_out.dim() < 1:
        raise ValueError("d_out must be [..., D]")
    D, N = d_out.shape[-1], int(N)
    if not isinstance(tokens, torch.Tensor):
        raise TypeError("tokens must be a torch.Tensor")
    _plain(tokens, "tokens", d_out.shape[:-1], torch.int64, dev)
    R = tokens.numel()
    with _on(stream, dev):
        ws, need = _workspace("rlscan_embed_tokens_workspace", dev, R, N, D)
        if d_table is None:
            d_table = torch.empty((N, D), dtype=dt, device=dev)
        else:
            _strided(d_table, "d_table", (N, D), dt, dev)
        _call("rlscan_embed_tokens_backward", _p._DTYPES[dt], d_out.data_ptr(), _table_rows(d_out, "d_out"),
              tokens.data_ptr(), d_table.data_ptr(), _table_rows(d_table, "d_table"), _ptr(ws), need, R, N, D,
              float(scale), _raw_stream(stream, dev))
    return d_table
