"""The policy operators: checks and marshalling for librlscan's linear attention,
action sampling and action log-probabilities (declared in include/rlscan.h).

Value tensors are float32, bfloat16 or float16, all of one dtype; states, decays,
uniform numbers, log-probabilities and entropies are float32.  Per-step tensors
may be strided (time-major, slices of a fused projection) as long as their last
dimension is contiguous.  Scratch memory and outputs that are not given are
allocated on the call's stream.  The functions are not differentiated by
autograd: each has its backward as a function of its own.
"""
from __future__ import annotations

import contextlib
import ctypes

import linear_recurrence_scan_reverse_amd as _rl

# Imported by the first call, like in the rest of the package, so that it loads without torch.
torch = None
_DTYPES = {}
_raw_stream_of = None


def _import_torch():
    global torch, _raw_stream_of
    import torch as module
    _DTYPES.update({module.float32: 0, module.bfloat16: 1, module.float16: 2})
    _raw_stream_of = module._C._cuda_getCurrentRawStream
    torch = module


class _Heads(ctypes.Structure):
    """rlscan_heads"""
    _fields_ = [("data", ctypes.c_void_p), ("env", ctypes.c_int64), ("step", ctypes.c_int64),
                ("head", ctypes.c_int64)]


_HEADS_BYTES = ctypes.sizeof(_Heads)
_ARRAYS = {n: ctypes.c_int64 * (4 * n) for n in (4, 7)}  # n rlscan_heads in a row


def _refuse(x, name, shape, dtype, device):
    """Raises for a tensor that _strided does not take."""
    if not isinstance(x, torch.Tensor):
        raise TypeError("%s must be a torch.Tensor" % name)
    if x.dtype != dtype:
        raise TypeError("%s must be %s, got %s" % (name, str(dtype).replace("torch.", ""), x.dtype))
    if x.shape != shape:
        raise ValueError("%s must have shape %s, got %s" % (name, tuple(shape), tuple(x.shape)))
    if x.device != device:
        raise ValueError("%s is on %s, expected %s" % (name, x.device, device))
    raise ValueError("%s must be contiguous in its last dimension" % name)


def _strided(x, name, shape, dtype, device):
    """A value tensor of any strides with a contiguous last dimension."""
    if not (isinstance(x, torch.Tensor) and x.dtype is dtype and x.shape == shape and x.device == device
            and (x.stride(-1) == 1 if shape else True) or _single(x, shape, dtype, device)):
        _refuse(x, name, shape, dtype, device)
    return x


def _single(x, shape, dtype, device):
    """Whether only the stride of a last dimension of one element was in the way."""
    return (isinstance(x, torch.Tensor) and x.dtype is dtype and x.shape == shape and x.device == device
            and shape[-1] <= 1)


def _plain(x, name, shape, dtype, device):
    """A contiguous tensor of the given dtype, or None."""
    if x is None:
        return None
    if not (isinstance(x, torch.Tensor) and x.dtype is dtype and x.shape == shape and x.device == device
            and x.is_contiguous()):
        _strided(x, name, shape, dtype, device)
        raise ValueError("%s must be contiguous" % name)
    return x


def _values(x, name, dims):
    if torch is None:
        _import_torch()
    if not isinstance(x, torch.Tensor):
        raise TypeError("%s must be a torch.Tensor" % name)
    if x.dim() != dims:
        raise ValueError("%s must have %d dimensions, got shape %s" % (name, dims, tuple(x.shape)))
    if x.dtype not in _DTYPES:
        raise TypeError("%s must be float32, bfloat16 or float16, got %s" % (name, x.dtype))
    return x


def _flags(x, name, shape, device):
    return None if x is None else _rl._check_flags(x, name, shape, device)


def _on_gpu(x, name):
    if not x.is_cuda:
        raise ValueError("%s must be on a GPU device, got %s" % (name, x.device))
    return x.device


_HERE = contextlib.nullcontext()


def _on(stream, device):
    """Allocations and launches go to the caller's stream, on the tensors' device."""
    if stream is not None:
        return torch.cuda.stream(stream)
    if device.index != torch._C._cuda_getDevice():
        return torch.cuda.device(device)
    return _HERE


def _raw_stream(stream, device):
    return _raw_stream_of(device.index) if stream is None else stream.cuda_stream


def _heads(tensors, time_major):
    """(array to keep alive, address) of the [E, T, heads, D] views of the tensors, one after the other."""
    v = []
    for x in tensors:
        s0, s1, s2, _ = x.stride()
        v += (x.data_ptr(), s1, s0, s2) if time_major else (x.data_ptr(), s0, s1, s2)
    a = _ARRAYS[len(tensors)](*v)
    return a, ctypes.addressof(a)


def _ptr(x):
    return None if x is None else x.data_ptr()


_functions = {}


def _call(fname, *args):
    fn = _functions.get(fname)
    if fn is None:
        fn = _functions[fname] = getattr(_rl.lib(), fname)
    st = fn(*args)
    if st != 0:
        raise _rl.RlscanError(st, fname)


def _workspace(fname, device, *sizes):
    """(tensor or None, bytes) of scratch memory that an entry asks for."""
    fn = _functions.get(fname)
    if fn is None:
        fn = _functions[fname] = getattr(_rl.lib(), fname)
    need = fn(*sizes)
    if need < 0:
        raise _rl.RlscanError(2, fname)
    return (torch.empty(need, dtype=torch.uint8, device=device) if need else None), need


def _scale(scale, K):
    """The given one or K^-0.5 (heads of no size are refused by the entry)."""
    return max(K, 1) ** -0.5 if scale is None else float(scale)


def _attention_inputs(q, k, v, log_decay, done, init_state, time_major):
    """Checks the inputs shared by the forward and the backward call."""
    _values(q, "q", 4)
    dev, dt = _on_gpu(q, "q"), q.dtype
    n0, n1, H, K = q.shape
    E, T = (n1, n0) if time_major else (n0, n1)
    for x, name in ((k, "k"), (v, "v")):
        _values(x, name, 4)
    Hkv, V = k.shape[2], v.shape[3]
    if H and (Hkv < 1 or H % Hkv):
        raise ValueError("q has %d heads, which is not a multiple of k's %d" % (H, Hkv))
    _strided(q, "q", q.shape, dt, dev)
    _strided(k, "k", (n0, n1, Hkv, K), dt, dev)
    _strided(v, "v", (n0, n1, Hkv, V), dt, dev)
    if not isinstance(log_decay, torch.Tensor):
        raise TypeError("log_decay must be a torch.Tensor")
    per_step = log_decay.dim() == 3
    _plain(log_decay, "log_decay", (n0, n1, H) if per_step else (H,), torch.float32, dev)
    done = _flags(done, "done", (n0, n1), dev)
    _plain(init_state, "init_state", (E, H, K, V), torch.float32, dev)
    return dev, dt, E, T, H, Hkv, K, V, per_step, done


def linear_attention(q, k, v, log_decay, done=None, init_state=None, *, scale=None, time_major=False,
                     with_state=False, out=None, final_state=None, stream=None):
    """Linear attention with a decay for each head, over whole rows.

    Per row and head S_t = exp(g_t) S_{t-1} + k_t v_t^T and o_t = scale * S_t^T q_t; the
    step after one flagged in ``done`` starts from a zero state, whatever the one before
    it held: inf and NaN stay within their episode.

    q [E, T, H, K], k [E, T, Hkv, K], v [E, T, Hkv, V] (``time_major``: [T, E, ...]),
    H a multiple of Hkv, K and V up to 128; log_decay: g, float32, [H] or [E, T, H];
    done [E, T]; init_state [E, H, K, V] float32; scale: K^-0.5 if not given.
    Returns out [E, T, H, V], or (out, final_state) with ``with_state`` or
    ``final_state``; final_state is what the next window takes as init_state."""
    dev, dt, E, T, H, Hkv, K, V, per_step, done = _attention_inputs(q, k, v, log_decay, done, init_state, time_major)
    shape = (q.shape[0], q.shape[1], H, V)
    scale = _scale(scale, K)
    fmt = _DTYPES[dt]
    with _on(stream, dev):
        out = torch.empty(shape, dtype=dt, device=dev) if out is None else _strided(out, "out", shape, dt, dev)
        if final_state is not None:
            _plain(final_state, "final_state", (E, H, K, V), torch.float32, dev)
        elif with_state:
            final_state = torch.empty((E, H, K, V), dtype=torch.float32, device=dev)
        ws, need = _workspace("rlscan_linear_attention_workspace", dev, fmt, E, T, H, Hkv, K, V, 0)
        keep, h = _heads((q, k, v, out), time_major)
        n = _HEADS_BYTES
        _call("rlscan_linear_attention", fmt, 1 if time_major else 0, h, h + n, h + 2 * n, log_decay.data_ptr(),
              per_step, _ptr(done), _ptr(init_state), h + 3 * n, _ptr(final_state), _ptr(ws), need, E, T, H, Hkv, K, V,
              scale, _raw_stream(stream, dev))
    return out if final_state is None else (out, final_state)


def linear_attention_backward(d_out, q, k, v, log_decay, done=None, init_state=None, d_final_state=None, *,
                              scale=None, time_major=False, dq=None, dk=None, dv=None, d_log_decay=None,
                              d_init_state=None, stream=None):
    """Gradients of ``linear_attention``: (dq, dk, dv, d_log_decay, d_init_state).

    d_out like the output; the other inputs as in the forward call; d_final_state
    [E, H, K, V], if the final state was used.  Gradients have the shapes of what they
    belong to (dk and dv are summed over the heads of a group); d_init_state is None
    without init_state."""
    dev, dt, E, T, H, Hkv, K, V, per_step, done = _attention_inputs(q, k, v, log_decay, done, init_state, time_major)
    _strided(d_out, "d_out", (q.shape[0], q.shape[1], H, V), dt, dev)
    _plain(d_final_state, "d_final_state", (E, H, K, V), torch.float32, dev)
    scale = _scale(scale, K)
    fmt = _DTYPES[dt]
    with _on(stream, dev):
        def grad(x, name, like):
            return torch.empty(like.shape, dtype=dt, device=dev) if x is None else _strided(x, name, like.shape, dt, dev)

        dq, dk, dv = grad(dq, "dq", q), grad(dk, "dk", k), grad(dv, "dv", v)
        if d_log_decay is None:
            d_log_decay = torch.empty_like(log_decay)
        else:
            _plain(d_log_decay, "d_log_decay", log_decay.shape, torch.float32, dev)
        if d_init_state is not None:
            _plain(d_init_state, "d_init_state", (E, H, K, V), torch.float32, dev)
        elif init_state is not None:
            d_init_state = torch.empty_like(init_state)
        ws, need = _workspace("rlscan_linear_attention_workspace", dev, fmt, E, T, H, Hkv, K, V, 1)
        keep, h = _heads((d_out, q, k, v, dq, dk, dv), time_major)
        h = [h + i * _HEADS_BYTES for i in range(7)]
        _call("rlscan_linear_attention_backward", fmt, 1 if time_major else 0, *h[:4], log_decay.data_ptr(), per_step,
              _ptr(done), _ptr(init_state), _ptr(d_final_state), *h[4:], d_log_decay.data_ptr(), _ptr(d_init_state),
              _ptr(ws), need, E, T, H, Hkv, K, V, scale, _raw_stream(stream, dev))
    return dq, dk, dv, d_log_decay, d_init_state


def linear_attention_step(q, k, v, log_decay, state, reset=None, slots=None, *, scale=None, out=None, stream=None):
    """One step of ``linear_attention`` for E rows; ``state`` is updated in place.

    q [E, H, K], k [E, Hkv, K], v [E, Hkv, V]; log_decay float32, [H] or [E, H]; state
    [S, H, K, V] float32; reset [E]: rows that start a new episode (their state is
    dropped unread); slots [E] int32: row e's state is state[slots[e]] (state[e] if
    not given).  A row whose slot is outside [0, S) gets zeros and changes nothing;
    two rows of a call must not share a slot.  Returns out [E, H, V]."""
    _values(q, "q", 3)
    dev, dt = _on_gpu(q, "q"), q.dtype
    E, H, K = q.shape
    for x, name in ((k, "k"), (v, "v")):
        _values(x, name, 3)
    Hkv, V = k.shape[1], v.shape[2]
    if H and (Hkv < 1 or H % Hkv):
        raise ValueError("q has %d heads, which is not a multiple of k's %d" % (H, Hkv))
    _strided(q, "q", q.shape, dt, dev)
    _strided(k, "k", (E, Hkv, K), dt, dev)
    _strided(v, "v", (E, Hkv, V), dt, dev)
    if not isinstance(log_decay, torch.Tensor):
        raise TypeError("log_decay must be a torch.Tensor")
    per_row = log_decay.dim() == 2
    _plain(log_decay, "log_decay", (E, H) if per_row else (H,), torch.float32, dev)
    if not isinstance(state, torch.Tensor) or state.dim() != 4:
        raise ValueError("state must be a [S, H, K, V] tensor")
    S = state.shape[0]
    _plain(state, "state", (S, H, K, V), torch.float32, dev)
    reset = _flags(reset, "reset", (E,), dev)
    _plain(slots, "slots", (E,), torch.int32, dev)
    if slots is None and S < E:
        raise ValueError("state has %d slots for %d rows" % (S, E))
    scale = _scale(scale, K)
    with _on(stream, dev):
        out = torch.empty((E, H, V), dtype=dt, device=dev) if out is None else _strided(out, "out", (E, H, V), dt, dev)
        v_ = []
        for x in (q, k, v, out):
            s0, s1, _ = x.stride()
            v_ += (x.data_ptr(), s0, 0, s1)
        keep = _ARRAYS[4](*v_)
        h, n = ctypes.addressof(keep), _HEADS_BYTES
        _call("rlscan_linear_attention_step", _DTYPES[dt], h, h + n, h + 2 * n, log_decay.data_ptr(), per_row,
              _ptr(reset), _ptr(slots), state.data_ptr(), h + 3 * n, E, S, H, Hkv, K, V, scale,
              _raw_stream(stream, dev))
    return out


def _logit_rows(logits, name="logits"):
    if torch is None:
        _import_torch()
    if not isinstance(logits, torch.Tensor):
        raise TypeError("%s must be a torch.Tensor" % name)
    if logits.dim() < 1 or logits.shape[-1] < 1:
        raise ValueError("%s must be [..., N] with N >= 1, got shape %s" % (name, tuple(logits.shape)))
    if logits.dtype not in _DTYPES:
        raise TypeError("%s must be float32, bfloat16 or float16, got %s" % (name, logits.dtype))
    return logits.shape[:-1], logits.numel() // logits.shape[-1], logits.shape[-1]


def _row_stride(x, name):
    """Elements between the rows of [..., N] taken in order."""
    N = x.shape[-1]
    if x.is_contiguous():
        return N
    if N > 1 and x.stride(-1) != 1:
        raise ValueError("%s must be contiguous in its last dimension" % name)
    step = None  # every leading dimension has to continue the one inside it
    for n, s in zip(reversed(x.shape[:-1]), reversed(x.stride()[:-1])):
        if n == 1:
            continue
        if step is None:
            first, step = s, s * n
        elif s == step:
            step = s * n
        else:
            raise ValueError("the rows of %s must lie at one distance" % name)
    return N if step is None else first


def _setting(x, name, shape, dtype, device, off):
    """(tensor, 0) for a row's own settings, (None, value) for one of all rows."""
    if isinstance(x, torch.Tensor):
        return _plain(x, name, shape, dtype, device), off
    return None, off if x is None else x


def _int32(x):
    """The nearest int32 to a whole number, so that one past the range stays refused, or off."""
    return max(-2 ** 31, min(int(x), 2 ** 31 - 1))


def sample_actions(logits, uniforms, *, temperature=1.0, top_k=None, top_p=None, min_p=None, mask=None, actions=None,
                   log_probs=None, stream=None):
    """One action for each row of logits [..., N], from uniform numbers in [0, 1).

    Keeps the top_k largest legal logits, of those the shortest prefix with top_p of
    their probability, and of those the ones with at least min_p of the largest one's
    probability, all after dividing by the temperature, then inverts the running sum in
    the order of the indices.  temperature, top_k, top_p and min_p are numbers or tensors
    [...] (top_k int32, the others float32); None, top_k 0, top_p 1 and min_p 0 are
    off; temperature 0 takes the largest logit.  mask [..., N]: zero where an action is
    not legal, nor are logits of -inf and NaN; +inf counts as the largest float32.
    Returns (actions int64 [...], log_probs float32 [...]): -1 and 0 for a row without
    a legal action."""
    lead, R, N = _logit_rows(logits)
    dev = _on_gpu(logits, "logits")
    stride = _row_stride(logits, "logits")
    if not isinstance(uniforms, torch.Tensor):
        raise TypeError("uniforms must be a torch.Tensor")
    _plain(uniforms, "uniforms", lead, torch.float32, dev)
    mask = _flags(mask, "mask", logits.shape, dev)
    temps, t1 = _setting(temperature, "temperature", lead, torch.float32, dev, 1.0)
    ks, k1 = _setting(top_k, "top_k", lead, torch.int32, dev, 0)
    ps, p1 = _setting(top_p, "top_p", lead, torch.float32, dev, 1.0)
    ms, m1 = _setting(min_p, "min_p", lead, torch.float32, dev, 0.0)
    with _on(stream, dev):
        if actions is None:
            actions = torch.empty(lead, dtype=torch.int64, device=dev)
        else:
            _plain(actions, "actions", lead, torch.int64, dev)
        if log_probs is None:
            log_probs = torch.empty_like(uniforms)
        else:
            _plain(log_probs, "log_probs", lead, torch.float32, dev)
        ws, need = _workspace("rlscan_sample_actions_workspace", dev, R, N)
        _call("rlscan_sample_actions_shared", _DTYPES[logits.dtype], logits.data_ptr(), stride, _ptr(mask),
              uniforms.data_ptr(), _ptr(temps), _ptr(ks), _ptr(ps), _ptr(ms), float(t1), _int32(k1),
              float(p1), float(m1), actions.data_ptr(), log_probs.data_ptr(), _ptr(ws), need, R, N,
              _raw_stream(stream, dev))
    return actions, log_probs


def action_log_probs(logits, actions, *, temperature=1.0, mask=None, log_probs=None, entropies=None, lse=None,
                     stream=None):
    """Log-probability of the taken action and entropy of softmax(logits / temperature).

    logits [..., N], actions [...] int64 (one outside [0, N), as for a padded step, has
    log-probability 0 and no gradient), mask [..., N]: zero where an action is not legal,
    as one with a logit of -inf (illegal taken ones: log-probability -inf).
    Returns (log_probs, entropies, lse) [...]: float32, and lse in float64 for the backward call."""
    lead, R, N = _logit_rows(logits)
    dev = _on_gpu(logits, "logits")
    stride = _row_stride(logits, "logits")
    if not isinstance(actions, torch.Tensor):
        raise TypeError("actions must be a torch.Tensor")
    _plain(actions, "actions", lead, torch.int64, dev)
    mask = _flags(mask, "mask", logits.shape, dev)
    with _on(stream, dev):
        outs = [torch.empty(lead, dtype=dt, device=dev) if x is None else _plain(x, name, lead, dt, dev)
                for x, name, dt in ((log_probs, "log_probs", torch.float32), (entropies, "entropies", torch.float32),
                                    (lse, "lse", torch.float64))]
        ws, need = _workspace("rlscan_action_log_probs_workspace", dev, R, N)
        _call("rlscan_action_log_probs", _DTYPES[logits.dtype], logits.data_ptr(), stride, _ptr(mask),
                  actions.data_ptr(), float(temperature), outs[0].data_ptr(), outs[1].data_ptr(), outs[2].data_ptr(),
                  _ptr(ws), need, R, N, _raw_stream(stream, dev))
    return tuple(outs)


def action_log_probs_backward(d_log_probs, d_entropies, logits, actions, lse, entropies, *, temperature=1.0, mask=None,
                              d_logits=None, stream=None):
    """Gradient of the logits of ``action_log_probs``, of their shape and dtype.

    d_log_probs and d_entropies [...] float32, either may be None; lse and entropies
    are the forward call's."""
    lead, R, N = _logit_rows(logits)
    dev = _on_gpu(logits, "logits")
    stride = _row_stride(logits, "logits")
    for x, name, dt in ((actions, "actions", torch.int64), (lse, "lse", torch.float64),
                        (entropies, "entropies", torch.float32)):
        if not isinstance(x, torch.Tensor):
            raise TypeError("%s must be a torch.Tensor" % name)
        _plain(x, name, lead, dt, dev)
    _plain(d_log_probs, "d_log_probs", lead, torch.float32, dev)
    _plain(d_entropies, "d_entropies", lead, torch.float32, dev)
    mask = _flags(mask, "mask", logits.shape, dev)
    with _on(stream, dev):
        if d_logits is None:
            d_logits = torch.empty(logits.shape, dtype=logits.dtype, device=dev)
        else:
            _strided(d_logits, "d_logits", logits.shape, logits.dtype, dev)
        _call("rlscan_action_log_probs_backward", _DTYPES[logits.dtype], _ptr(d_log_probs), _ptr(d_entropies),
                  logits.data_ptr(), stride, _ptr(mask), actions.data_ptr(), float(temperature), lse.data_ptr(),
                  entropies.data_ptr(), d_logits.data_ptr(), _row_stride(d_logits, "d_logits"), R, N,
                  _raw_stream(stream, dev))
    return d_logits
