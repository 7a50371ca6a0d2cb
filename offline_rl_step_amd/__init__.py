"""Python binding of libiqlher.so, the MI355X IQL + HER step.

Argument marshalling only: every function forwards to the C entry point of
the same name in ``include/iqlher.h``; tensors are passed by ``data_ptr()``
and the work is enqueued on torch's current HIP stream.  There is no CPU or
PyTorch fallback: importing this module fails loudly when the library has not
been built (``python offline_rl_step_amd/build.py``).
"""
import bisect
import ctypes
import os

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libiqlher.so")

# torch owns device memory and streams; importing it first makes the library
# bind to the same HIP runtime instance.
import torch  # noqa: E402,F401

if not os.path.exists(LIB_PATH):
    raise ImportError(f"{LIB_PATH} is missing: build it with `python offline_rl_step_amd/build.py`")
_lib = ctypes.CDLL(LIB_PATH)

OK, EINVAL, ESHAPE, ENOMEM, EHIP, ENONFINITE = 0, -1, -2, -3, -4, -5
F32, BF16, F16 = 0, 1, 2
NORM_L2, NORM_MAX = 0, 1
HER_FINAL, HER_FUTURE, HER_RANDOM = 0, 1, 2
FLAG_NONFINITE_GRAD, FLAG_BAD_INDEX, FLAG_NONFINITE_LOSS, FLAG_NONFINITE_STATE = 0x1, 0x2, 0x4, 0x8
MAX_SOURCES = 8

_p = ctypes.c_void_p
_i32, _i64, _u64, _f = ctypes.c_int32, ctypes.c_int64, ctypes.c_uint64, ctypes.c_float


class IqlConfig(ctypes.Structure):
    _fields_ = [("state_dim", _i32), ("hidden", _i32), ("max_batch", _i32), ("num_groups", _i32),
                ("compute_dtype", _i32), ("hidden2", _i32), ("states_ld", _i64),
                ("tau", _f * 2), ("lr", _f), ("beta1", _f), ("beta2", _f), ("eps", _f),
                ("weight_decay", _f), ("max_grad_norm", _f), ("weight_clamp_max_abs", _f)]


class HerConfig(ctypes.Structure):
    _fields_ = [("state_dim", _i32), ("goal_dim", _i32), ("strategy", _i32), ("reserved0", _i32),
                ("goal_threshold", _f), ("reward_hit", _f), ("reward_miss", _f), ("reserved1", _f)]


class HerBuffer(ctypes.Structure):
    _fields_ = [("states", _p), ("next_states", _p), ("actions", _p), ("rewards", _p), ("dones", _p),
                ("episode_ends", _p), ("capacity", _i64), ("buffer_size", _i64),
                ("num_episodes", _i32), ("reserved0", _i32)]


class HerOut(ctypes.Structure):
    _fields_ = [("donor_idx", _p), ("states", _p), ("states_dtype", _i32), ("reserved0", _i32),
                ("states_ld", _i64), ("next_states", _p), ("actions", _p), ("rewards", _p),
                ("dones", _p), ("d_flags", _p), ("is_weights", _p)]


class Adam(ctypes.Structure):
    _fields_ = [("params", _p), ("m", _p), ("v", _p), ("t", _p), ("d_flags", _p),
                ("lr", _f), ("beta1", _f), ("beta2", _f), ("eps", _f), ("weight_decay", _f),
                ("max_grad_norm", _f), ("weight_clamp_max_abs", _f), ("reserved0", _f)]


class HerStep(ctypes.Structure):
    _fields_ = [("cfg", ctypes.POINTER(HerConfig)), ("buf", ctypes.POINTER(HerBuffer)), ("source_idx", _p),
                ("out", ctypes.POINTER(HerOut)), ("seed", _u64), ("n", _i32), ("reserved0", _i32)]


class BudgetStep(ctypes.Structure):
    _fields_ = [("grad_buf", _p), ("sources", ctypes.POINTER(_p)), ("fractions", ctypes.POINTER(_f)),
                ("alphas", ctypes.POINTER(_f)), ("out_norms", _p), ("adam", ctypes.POINTER(Adam)),
                ("workspace", _p), ("workspace_bytes", ctypes.c_size_t), ("n", _i64), ("num_sources", _i32),
                ("max_grad_norm", _f)]


class TensorSetStruct(ctypes.Structure):
    _fields_ = [("d_table", _p), ("table_bytes", ctypes.c_size_t), ("numel", _i64), ("count", _i32),
                ("pieces", _i32), ("overlap", _i32), ("reserved0", _i32)]


class Mx4Struct(ctypes.Structure):
    _fields_ = [("codes", _p), ("scales", _p), ("rows", _i64), ("cols", _i64)]


def _sig(name, res, args):
    fn = getattr(_lib, name)
    fn.restype = res
    fn.argtypes = args
    return fn


_lib_iql_num_params = _sig("iql_num_params", _i32, [_i32, _i32, ctypes.POINTER(_i64)])
_lib_iql_config_num_params = _sig("iql_config_num_params", _i32, [ctypes.POINTER(IqlConfig), ctypes.POINTER(_i64)])
_lib_iql_create = _sig("iql_create", _i32, [ctypes.POINTER(IqlConfig), _p, ctypes.POINTER(_p)])
_lib_iql_destroy = _sig("iql_destroy", _i32, [_p])
_lib_iql_train_step = _sig("iql_train_step", _i32, [_p, _p, _p, _i32, _p, _p, _p, _p])
_lib_iql_train_step_aw = _sig("iql_train_step_aw", _i32, [_p, _p, _p, _i32, _p, _i32, _f, _p, _p, _p, _p, _p])
_lib_iql_compute_gradients = _sig("iql_compute_gradients", _i32, [_p, _p, _p, _i32, _p, _p])
_lib_iql_apply_gradients = _sig("iql_apply_gradients", _i32, [_p, _i32, _p, _p, _p])
_lib_iql_time_cg = _sig("iql_time_compute_gradients", _i32, [_p, _p, _p, _i32, _i32, ctypes.POINTER(_f), _p])
_lib_iql_partial_layout = _sig("iql_partial_layout", _i32, [_p, _i32, ctypes.POINTER(_i32), ctypes.POINTER(_i64)])
_lib_iql_get_state = _sig("iql_get_state", _i32, [_p, _i32, _p, _p, _p, _p, _p])
_lib_iql_set_state = _sig("iql_set_state", _i32, [_p, _i32, _p, _p, _p, _p, _p])
_lib_iql_forward_values = _sig("iql_forward_values", _i32, [_p, _p, _i32, _i64, _i32, _p, _p, _p, _f, _p, _p])
_lib_iql_target_ema_update = _sig("iql_target_ema_update", _i32, [_p, _f, _p])
_lib_iql_set_target_ema = _sig("iql_set_target_ema", _i32, [_p, _f])
_lib_iql_get_target = _sig("iql_get_target", _i32, [_p, _i32, _p, _p])
_lib_iql_set_target = _sig("iql_set_target", _i32, [_p, _i32, _p, _p])
_lib_iql_step_counter = _sig("iql_step_counter", _p, [_p])
_lib_iql_flags = _sig("iql_flags", _p, [_p])
_lib_iql_status = _sig("iql_status", _i32, [_p, ctypes.POINTER(_i32)])
_lib_iql_aw_policy = _sig("iql_aw_policy", _i32, [_p, _p, _i32, _i32, _i32, _f, _p, _p])
_lib_her_relabel = _sig("her_relabel", _i32, [ctypes.POINTER(HerConfig), ctypes.POINTER(HerBuffer), _p, _i32,
                                              _u64, _p, ctypes.POINTER(HerOut), _p])
_lib_ws_bytes = _sig("grad_budget_workspace_bytes", _i32, [_i64, _i32, ctypes.POINTER(ctypes.c_size_t)])
_lib_budget = _sig("grad_budget_accumulate", _i32, [_p, ctypes.POINTER(_p), ctypes.POINTER(_f),
                                                    ctypes.POINTER(_f), _i32, _i64, _f, _p,
                                                    ctypes.POINTER(Adam), _p, ctypes.c_size_t, _p])
_lib_budget_noalloc = _sig("grad_budget_accumulate_noalloc", _i32, [_p, ctypes.POINTER(_p), ctypes.POINTER(_f),
                                                                    ctypes.POINTER(_f), _i32, _i64, _f, _p,
                                                                    ctypes.POINTER(Adam), _p])
_lib_iql_aux_step = _sig("iql_aux_step", _i32, [_p, ctypes.POINTER(HerStep), _p, _p, _i32, _p, _i32, _f, _p, _p,
                                                _p, _p, ctypes.POINTER(BudgetStep), _p])
_lib_iql_time_aux_step = _sig("iql_time_aux_step", _i32, [_p, ctypes.POINTER(HerStep), _p, _p, _i32, _p, _i32, _f,
                                                          _p, _p, _p, _p, ctypes.POINTER(BudgetStep), _i32,
                                                          ctypes.POINTER(_f), _p])
_lib_iql_aux_step_phase_stamps = _sig("iql_aux_step_phase_stamps", _i32,
                                      [_p, ctypes.POINTER(HerStep), _p, _p, _i32, _p, _i32, _f, _p, _p, _p, _p,
                                       ctypes.POINTER(BudgetStep), _p, _i32, _p])
_lib_per_ws = _sig("per_workspace_bytes", _i32, [_i64, ctypes.POINTER(ctypes.c_size_t)])
_lib_per_sample = _sig("per_sample_indices", _i32, [_p, _i64, _i32, _u64, _p, _f, _p, _p, _p, _p, ctypes.c_size_t, _p])
_lib_nonfinite_check = _sig("iqlh_nonfinite_check", _i32, [ctypes.POINTER(_p), ctypes.POINTER(_i64), _i32, _p, _p])
_lib_set_bytes = _sig("iqlh_tensor_set_bytes", _i32, [ctypes.POINTER(_i64), ctypes.POINTER(_i32), _i32,
                                                      ctypes.POINTER(ctypes.c_size_t)])
_lib_set_fill = _sig("iqlh_tensor_set_fill", _i32, [ctypes.POINTER(_p), ctypes.POINTER(_i64), ctypes.POINTER(_i32),
                                                    _i32, _p, ctypes.c_size_t, ctypes.POINTER(TensorSetStruct)])
_lib_norm_ws = _sig("iqlh_grad_norm_workspace_bytes", _i32, [ctypes.POINTER(TensorSetStruct),
                                                             ctypes.POINTER(ctypes.c_size_t)])
_lib_grad_norm = _sig("iqlh_grad_norm", _i32, [ctypes.POINTER(TensorSetStruct), _i32, _p, _p, _p, _p,
                                               ctypes.c_size_t, _p])
_lib_grad_clip = _sig("iqlh_grad_clip", _i32, [ctypes.POINTER(TensorSetStruct), _i32, ctypes.c_double, _p, _p, _p, _p,
                                               ctypes.c_size_t, _p])
_lib_mx4_quantize = _sig("iqlh_mx4_quantize", _i32, [_p, _i32, _i64, _i32, ctypes.POINTER(Mx4Struct), _p])
_lib_mx4_dequantize = _sig("iqlh_mx4_dequantize", _i32, [ctypes.POINTER(Mx4Struct), _p, _i32, _i64, _p])
_lib_mx4_ws = _sig("iqlh_mx4_workspace_bytes", _i32, [_i64, _i64, _i64, ctypes.POINTER(ctypes.c_size_t)])
_lib_mx4_matmul = _sig("iqlh_mx4_matmul", _i32, [ctypes.POINTER(Mx4Struct), ctypes.POINTER(Mx4Struct), _p, _i32, _p,
                                                 _i32, _i64, _p, ctypes.c_size_t, _p])
_lib_mx4_linear = _sig("iqlh_mx4_linear", _i32, [_p, _i32, _i64, _i64, ctypes.POINTER(Mx4Struct), _p, _i32, _p, _i32,
                                                 _i64, _p, ctypes.c_size_t, _p])
_lib_forward_mx4_ws = _sig("iql_forward_values_mx4_workspace_bytes", _i32, [_p, _i32,
                                                                            ctypes.POINTER(ctypes.c_size_t)])
_lib_forward_mx4 = _sig("iql_forward_values_mx4", _i32, [_p, _p, _i32, _i64, _i32, _p, _p, _p, _f, _p, _p,
                                                         ctypes.c_size_t, _p])
_lib_last_error = _sig("iqlh_last_error", ctypes.c_char_p, [])


class IqlhError(RuntimeError):
    def __init__(self, code, where):
        self.code = code
        msg = _lib_last_error().decode(errors="replace")
        super().__init__(f"{where} failed with status {code}: {msg}")


def _check(code, where):
    if code != OK:
        raise IqlhError(code, where)
    return code


def _ptr(t):
    """Device (or host) address of a tensor, or None."""
    return None if t is None else ctypes.c_void_p(t.data_ptr())


# Current device and the handle of its current stream without building a
# Stream object (0.1 us each against 3 us, which is as long as a launch takes)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
_get_device = getattr(torch._C, "_cuda_getDevice", None)
if _get_device is None:
    _raw_stream, _get_device = None, torch.cuda.current_device


def _stream(stream):
    if stream is None:
        if _raw_stream is not None and torch.cuda.is_initialized():
            return ctypes.c_void_p(_raw_stream(_get_device()))
        return ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)
    if isinstance(stream, int):
        return ctypes.c_void_p(stream)
    return ctypes.c_void_p(stream.cuda_stream)


def _stream_object(stream, device):
    """torch's stream of an address.  ExternalStream takes 0, the default
    stream's, for none given and returns a stream of torch's pool."""
    return torch.cuda.ExternalStream(stream, device=device) if stream else torch.cuda.default_stream(device)


def _stream_of(stream, device_index, *tensors):
    """The call's stream as an address, where CUDA is known to be initialised.
    torch's allocator knows of the current stream only: for another one the
    memory of the call's tensors (or None) is kept until the call has run, should
    they be dropped before.  (Tensors of a captured call have to outlive the
    graph anyway.)"""
    if _raw_stream is not None:
        current = _raw_stream(device_index)
    else:
        current = torch.cuda.current_stream().cuda_stream
    if stream is None:
        return current
    address = _stream(stream).value or 0
    if address != current and not torch.cuda.is_current_stream_capturing():
        other = _stream_object(address, device_index)
        for t in tensors:
            if t is not None:
                t.record_stream(other)
    return address


def last_error():
    return _lib_last_error().decode(errors="replace")


# ------------------------------------------------------------------- IQL
def iql_num_params(state_dim, hidden):
    out = _i64()
    _check(_lib_iql_num_params(state_dim, hidden, ctypes.byref(out)), "iql_num_params")
    return out.value


def iql_config_num_params(cfg):
    out = _i64()
    _check(_lib_iql_config_num_params(ctypes.byref(cfg), ctypes.byref(out)), "iql_config_num_params")
    return out.value


def make_config(state_dim, hidden, max_batch, num_groups=1, compute_dtype=F32, states_ld=None,
                tau=(0.7, 0.7), lr=3e-4, beta1=0.9, beta2=0.999, eps=1e-8, weight_decay=0.0,
                max_grad_norm=1.0, weight_clamp_max_abs=0.0, hidden2=0):
    """hidden: first hidden width H1; hidden2: second (0 = hidden)."""
    c = IqlConfig()
    c.state_dim, c.hidden, c.max_batch, c.num_groups = state_dim, hidden, max_batch, num_groups
    c.hidden2 = hidden2
    c.compute_dtype = compute_dtype
    c.states_ld = state_dim if states_ld is None else states_ld
    taus = list(tau) + [tau[-1]] * (2 - len(tau))
    c.tau[0], c.tau[1] = taus[0], taus[1]
    c.lr, c.beta1, c.beta2, c.eps = lr, beta1, beta2, eps
    c.weight_decay, c.max_grad_norm, c.weight_clamp_max_abs = weight_decay, max_grad_norm, weight_clamp_max_abs
    return c


def iql_create(cfg, init_params_host):
    """init_params_host: contiguous float32 host array/tensor of num_groups * P."""
    import numpy as np
    arr = np.ascontiguousarray(np.asarray(init_params_host, dtype=np.float32))
    h = _p()
    _check(_lib_iql_create(ctypes.byref(cfg), arr.ctypes.data_as(_p), ctypes.byref(h)), "iql_create")
    return h


def iql_destroy(h):
    _check(_lib_iql_destroy(h), "iql_destroy")


def iql_train_step(h, states, q_taken, batch, out_v=None, out_loss=None, out_grad_norm=None, stream=None):
    _check(_lib_iql_train_step(h, _ptr(states), _ptr(q_taken), batch, _ptr(out_v), _ptr(out_loss),
                               _ptr(out_grad_norm), _stream(stream)), "iql_train_step")


def iql_train_step_aw(h, states, q_taken, batch, q_all, num_actions, beta, out_pi, out_v, out_loss=None,
                      out_grad_norm=None, stream=None):
    _check(_lib_iql_train_step_aw(h, _ptr(states), _ptr(q_taken), batch, _ptr(q_all), num_actions, beta,
                                  _ptr(out_pi), _ptr(out_v), _ptr(out_loss), _ptr(out_grad_norm),
                                  _stream(stream)), "iql_train_step_aw")


def iql_compute_gradients(h, states, q_taken, batch, out_v=None, stream=None):
    _check(_lib_iql_compute_gradients(h, _ptr(states), _ptr(q_taken), batch, _ptr(out_v), _stream(stream)),
           "iql_compute_gradients")


def iql_apply_gradients(h, batch, out_loss=None, out_grad_norm=None, stream=None):
    _check(_lib_iql_apply_gradients(h, batch, _ptr(out_loss), _ptr(out_grad_norm), _stream(stream)),
           "iql_apply_gradients")


def iql_time_compute_gradients(h, states, q_taken, batch, reps, stream=None):
    """Mean duration (us) of the fused forward/backward kernel over `reps` launches."""
    out = _f()
    _check(_lib_iql_time_cg(h, _ptr(states), _ptr(q_taken), batch, reps, ctypes.byref(out), _stream(stream)),
           "iql_time_compute_gradients")
    return out.value


def iql_partial_layout(h, batch):
    """(partial rows per group, floats per row) of the per-workgroup gradient
    partials written for `batch` rows."""
    rows, floats = _i32(), _i64()
    _check(_lib_iql_partial_layout(h, batch, ctypes.byref(rows), ctypes.byref(floats)), "iql_partial_layout")
    return rows.value, floats.value


def per_workspace_bytes(size):
    out = ctypes.c_size_t()
    _check(_lib_per_ws(size, ctypes.byref(out)), "per_workspace_bytes")
    return out.value


def per_sample_indices(priorities, n, seed, beta, out_idx, out_weights, workspace, d_step=None, d_flags=None,
                       stream=None):
    """n prioritized draws over the rows of `priorities` (f32 tensor)."""
    _check(_lib_per_sample(_ptr(priorities), priorities.numel(), n, seed, _ptr(d_step), beta, _ptr(out_idx),
                           _ptr(out_weights), _ptr(d_flags), _ptr(workspace),
                           workspace.numel() * workspace.element_size(), _stream(stream)), "per_sample_indices")


def nonfinite_check(buffers, slot_flags, stream=None):
    """Sets slot_flags[s] = 1 for every buffer (fp32 tensor or None) holding
    a NaN or an infinity; clean slots keep their value."""
    n = len(buffers)
    ptrs = (_p * n)(*[None if b is None else b.data_ptr() for b in buffers])
    lens = (_i64 * n)(*[0 if b is None else b.numel() for b in buffers])
    _check(_lib_nonfinite_check(ptrs, lens, n, _ptr(slot_flags), _stream(stream)), "iqlh_nonfinite_check")


def iql_forward_values(h, next_states, batch, out_v, rewards=None, dones=None, gamma=0.99, out_target=None,
                       states_ld=None, stream=None):
    """V(s') of every group (online parameters) and, with rewards, the
    bootstrap target r + gamma (1 - done) V(s')."""
    import torch
    dt = BF16 if next_states.dtype == torch.bfloat16 else F32
    ld = states_ld if states_ld is not None else next_states.stride(0)
    _check(_lib_iql_forward_values(h, _ptr(next_states), dt, ld, batch, _ptr(out_v), _ptr(rewards), _ptr(dones),
                                   gamma, _ptr(out_target), _stream(stream)), "iql_forward_values")


def iql_target_ema_update(h, tau, stream=None):
    _check(_lib_iql_target_ema_update(h, tau, _stream(stream)), "iql_target_ema_update")


def iql_set_target_ema(h, tau):
    _check(_lib_iql_set_target_ema(h, tau), "iql_set_target_ema")


def iql_get_target(h, group, params, stream=None):
    _check(_lib_iql_get_target(h, group, _ptr(params), _stream(stream)), "iql_get_target")


def iql_set_target(h, group, params, stream=None):
    _check(_lib_iql_set_target(h, group, _ptr(params), _stream(stream)), "iql_set_target")


def iql_get_state(h, group, params=None, m=None, v=None, t=None, stream=None):
    _check(_lib_iql_get_state(h, group, _ptr(params), _ptr(m), _ptr(v), _ptr(t), _stream(stream)),
           "iql_get_state")


def iql_set_state(h, group, params, m, v, t, stream=None):
    _check(_lib_iql_set_state(h, group, _ptr(params), _ptr(m), _ptr(v), _ptr(t), _stream(stream)),
           "iql_set_state")


def iql_step_counter(h):
    return _lib_iql_step_counter(h)


def iql_flags(h):
    return _lib_iql_flags(h)


def iql_status(h):
    """Returns (status, flags); synchronises the device."""
    f = _i32()
    rc = _lib_iql_status(h, ctypes.byref(f))
    return rc, f.value


def iql_aw_policy(q, v, num_groups, batch, num_actions, beta, out_pi, stream=None):
    _check(_lib_iql_aw_policy(_ptr(q), _ptr(v), num_groups, batch, num_actions, beta, _ptr(out_pi),
                              _stream(stream)), "iql_aw_policy")


# ----------------------------------------------- norm and clip of tensor lists
_DTYPES = {torch.float32: F32, torch.bfloat16: BF16, torch.float16: F16}


def _need(ok, what):
    if not ok:
        raise ValueError(what)


# The checks below run in every call: messages are built only when they fail.
def _float_code(t, what):
    code = _DTYPES.get(t.dtype)
    if code is None:
        raise ValueError(f"{what}: {t.dtype} is none of float32, bfloat16, float16")
    return code


def _need_f32(t, numel, device, what):
    """t: a contiguous float32 tensor of at least `numel` elements on `device`."""
    if not (t.dtype == torch.float32 and t.is_contiguous() and t.numel() >= numel and t.device == device):
        raise ValueError(f"{what} must be a contiguous float32 tensor of at least {numel} elements on {device}")


def _need_current(device):
    """The library enqueues on the current device; returns its index."""
    if device.type != "cuda":
        raise ValueError(f"tensors are on {device}: the kernels read device memory")
    index = _get_device()  # tensors on it exist, so CUDA is initialised
    if device.index != index:
        raise ValueError(f"tensors are on {device}, the current device is cuda:{index}")
    return index


class TensorSet:
    """The tensors of one network (float32, bfloat16, float16 in any mix, each
    contiguous, all on the current device), cut into pieces once for any number of
    grad_norm / grad_clip calls.  Keeps the tensors' memory and goes by it:
    gradients must stay where they are from step to step (cleared with
    ``set_to_none=False``; new ones need a new set, the old set's calls go on
    reading and clipping the old memory)."""

    def __init__(self, tensors):
        self.tensors = tensors = list(tensors)
        self._memory = [t.detach() for t in tensors]  # what the table's addresses lie in, should t.data be replaced
        _need(len(tensors) > 0, "TensorSet needs at least one tensor")
        self.device = tensors[0].device
        _need_current(self.device)
        for i, t in enumerate(tensors):
            _need(t.device == self.device, f"tensor {i} is on {t.device}, the first on {self.device}")
            _need(t.is_contiguous(), f"tensor {i} is not contiguous")
            _float_code(t, f"tensor {i}")
        k = len(tensors)
        ptrs = (_p * k)(*[t.data_ptr() or None for t in tensors])
        lens = (_i64 * k)(*[t.numel() for t in tensors])
        types = (_i32 * k)(*[_DTYPES[t.dtype] for t in tensors])
        need = ctypes.c_size_t()
        _check(_lib_set_bytes(lens, types, k, ctypes.byref(need)), "iqlh_tensor_set_bytes")
        host = torch.empty(need.value + 16, dtype=torch.uint8)
        lead = -host.data_ptr() % 16
        host = host[lead:lead + need.value]
        self.struct = TensorSetStruct()
        _check(_lib_set_fill(ptrs, lens, types, k, host.data_ptr(), need.value, ctypes.byref(self.struct)),
               "iqlh_tensor_set_fill")
        # a copy from pageable memory: complete when it returns, for any stream
        self.table = host[:self.struct.table_bytes].to(self.device)
        # the allocator reuses the table's memory in this stream's order
        self._streams = {_stream_of(None, self.device.index)}
        self.struct.d_table = self.table.data_ptr()
        self.ref = ctypes.byref(self.struct)
        self.numel, self.count = self.struct.numel, self.struct.count
        self._ranges = sorted((t.data_ptr(), t.data_ptr() + t.numel() * t.element_size()) for t in tensors if t.numel())

    def _used_on(self, stream):
        """`stream`, an address.  Keeps the memory of the table and the tensors from being handed out
        again, should the set be dropped, before the calls on another stream have read it."""
        if stream not in self._streams and not torch.cuda.is_current_stream_capturing():
            other = _stream_object(stream, self.device)
            for t in (self.table, *self._memory):
                t.record_stream(other)
            self._streams.add(stream)  # good until the memory is freed
        return stream

    def overlaps(self, t):
        """Whether t (contiguous) shares memory with a tensor of the set."""
        return self._overlaps_range(t.data_ptr(), t.data_ptr() + t.numel() * t.element_size())

    def _overlaps_range(self, lo, hi):
        if self.struct.overlap:  # ranges are not disjoint: look at each
            return any(a < hi and lo < b for a, b in self._ranges)
        i = bisect.bisect_left(self._ranges, (hi,))
        return any(a < hi and lo < b for a, b in self._ranges[max(0, i - 1):i])


def grad_norm_workspace(tensor_set):
    """A workspace for grad_norm / grad_clip calls on the set, on any stream (its counter is at 0 when this returns)."""
    out = ctypes.c_size_t()
    _check(_lib_norm_ws(ctypes.byref(tensor_set.struct), ctypes.byref(out)), "iqlh_grad_norm_workspace_bytes")
    ws = torch.empty(out.value, dtype=torch.uint8, device=tensor_set.device)
    if torch.cuda.is_current_stream_capturing():
        ws[:64].zero_()  # recorded in front of the graph's calls
    else:
        ws[:64].copy_(torch.zeros(64, dtype=torch.uint8))  # from pageable memory: complete when it returns, for any stream
    return ws


def _need_aux(device, workspace, flags):
    if workspace.device != device or not workspace.is_contiguous():
        raise ValueError(f"workspace must be contiguous on {device}")
    if flags is not None and (flags.dtype != torch.int32 or flags.device != device or flags.numel() < 1):
        raise ValueError(f"flags must be an int32 tensor on {device}")


def grad_norm(tensor_set, out_norm, workspace, kind=NORM_L2, out_each=None, flags=None, stream=None):
    """Norm over all tensors of the set into out_norm [1], with out_each
    [count] each tensor's own too."""
    s = tensor_set
    index = _need_current(s.device)
    _need_f32(out_norm, 1, s.device, "out_norm")
    if out_each is not None:
        _need_f32(out_each, s.count, s.device, "out_each")
    _need_aux(s.device, workspace, flags)
    _check(_lib_grad_norm(s.ref, kind, out_norm.data_ptr(), _ptr(out_each), _ptr(flags), workspace.data_ptr(),
                          workspace.nbytes, s._used_on(_stream_of(stream, index, out_norm, out_each, flags, workspace))),
           "iqlh_grad_norm")


def grad_clip(tensor_set, max_norm, out, workspace, kind=NORM_L2, out_flat=None, flags=None, stream=None):
    """Clips the set to max_norm: in place, or into the flat float32 vector
    out_flat [numel] with the tensors unchanged.  out [2]: norm and factor."""
    s = tensor_set
    index = _need_current(s.device)
    _need_f32(out, 2, s.device, "out")
    flat = None
    if out_flat is not None:
        _need_f32(out_flat, s.numel, s.device, "out_flat")
        flat = out_flat.data_ptr()
        _need(not s._overlaps_range(flat, flat + 4 * s.numel), "out_flat shares memory with a tensor of the set")
    _need_aux(s.device, workspace, flags)
    _check(_lib_grad_clip(s.ref, kind, max_norm, flat, out.data_ptr(), _ptr(flags), workspace.data_ptr(),
                          workspace.nbytes, s._used_on(_stream_of(stream, index, out, out_flat, flags, workspace))),
           "iqlh_grad_clip")


# --------------------------------------------- microscaled 4-bit matrices
class Mx4:
    """A matrix [rows, cols] in blocks of 32 elements along its rows: `codes`
    uint8 [rows, kb * 16] and `scales` uint8 [rows, kb], kb = ceil(cols / 32),
    both contiguous on one device."""

    def __init__(self, codes, scales, rows, cols):
        kb = -(-cols // 32)
        _need(codes.dtype == torch.uint8 and codes.is_contiguous() and codes.numel() == rows * kb * 16,
              f"codes must be contiguous uint8 of {rows} x {kb * 16}")
        _need(scales.dtype == torch.uint8 and scales.is_contiguous() and scales.numel() == rows * kb
              and scales.device == codes.device, f"scales must be contiguous uint8 of {rows} x {kb} beside the codes")
        self.codes, self.scales, self.rows, self.cols = codes, scales, rows, cols
        self.device = codes.device
        self.struct = Mx4Struct(codes.data_ptr(), scales.data_ptr(), rows, cols)
        self.ref = ctypes.byref(self.struct)


def mx4_empty(rows, cols, axis=1, device=None):
    """An Mx4 for mx4_quantize(x, .., axis) of x [rows, cols]; with axis 0 it
    holds the transpose, [cols, rows]."""
    _need(axis in (0, 1), "axis must be 0 or 1")
    if axis == 0:
        rows, cols = cols, rows
    kb = -(-cols // 32)
    device = torch.device("cuda", torch.cuda.current_device()) if device is None else device
    return Mx4(torch.empty((rows, kb * 16), dtype=torch.uint8, device=device),
               torch.empty((rows, kb), dtype=torch.uint8, device=device), rows, cols)


def _matrix(t, rows, cols, device, what):
    """(dtype code, row stride) of a [rows, cols] tensor with unit column stride."""
    if t.shape != (rows, cols) or t.device != device:
        raise ValueError(f"{what} must be [{rows}, {cols}] on {device}, is {list(t.shape)} on {t.device}")
    ld, step = t.stride()
    if (cols > 1 and step != 1) or (rows > 1 and ld < cols):
        raise ValueError(f"{what} must have neighbouring columns and rows that do not overlap")
    return _float_code(t, what), ld if rows > 1 else cols


def mx4_quantize(x, out, axis=1, stream=None):
    """Quantises x [rows, cols] (float32, bfloat16, float16; rows may be
    strided) in blocks along its rows (axis=1) or, transposed, its columns
    (axis=0) into the Mx4 `out`, which must not share memory with it."""
    if axis not in (0, 1):
        raise ValueError("axis must be 0 or 1")
    index = _need_current(out.device)
    r, c = (out.rows, out.cols) if axis == 1 else (out.cols, out.rows)
    dt, ld = _matrix(x, r, c, out.device, "x")
    _check(_lib_mx4_quantize(x.data_ptr(), dt, ld, 1 - axis, out.ref,
                             _stream_of(stream, index, x, out.codes, out.scales)), "iqlh_mx4_quantize")


def mx4_dequantize(q, out, stream=None):
    """Values of q into out [rows, cols] (float32, bfloat16, float16)."""
    index = _need_current(q.device)
    dt, ld = _matrix(out, q.rows, q.cols, q.device, "out")
    _check(_lib_mx4_dequantize(q.ref, out.data_ptr(), dt, ld, _stream_of(stream, index, q.codes, q.scales, out)),
           "iqlh_mx4_dequantize")


def mx4_matmul_workspace(m, n, k, device=None):
    """A workspace for mx4_matmul / mx4_linear calls of these sizes."""
    out = ctypes.c_size_t()
    _check(_lib_mx4_ws(m, n, k, ctypes.byref(out)), "iqlh_mx4_workspace_bytes")
    device = torch.device("cuda", torch.cuda.current_device()) if device is None else device
    return torch.empty(out.value, dtype=torch.uint8, device=device)


def _need_product(rows, b, out, workspace, bias):
    index = _need_current(b.device)
    _need_aux(b.device, workspace, None)
    if bias is not None:
        _need_f32(bias, b.rows, b.device, "bias")
    return *_matrix(out, rows, b.rows, b.device, "out"), index


def mx4_matmul(a, b, out, workspace, bias=None, relu=False, stream=None):
    """out[m, n] = act(sum_k a[m, k] b[n, k] + bias[n]) of two Mx4; out must not
    share memory with an operand."""
    if a.device != b.device:
        raise ValueError(f"a is on {a.device}, b on {b.device}")
    dt, ld, index = _need_product(a.rows, b, out, workspace, bias)
    _check(_lib_mx4_matmul(a.ref, b.ref, None if bias is None else bias.data_ptr(), int(relu), out.data_ptr(), dt, ld,
                           workspace.data_ptr(), workspace.nbytes,
                           _stream_of(stream, index, a.codes, a.scales, b.codes, b.scales, bias, out, workspace)),
           "iqlh_mx4_matmul")


def mx4_linear(x, b, out, workspace, bias=None, relu=False, stream=None):
    """mx4_matmul with a = x [m, k] (float32, bfloat16, float16) quantised on the way."""
    rows = x.shape[0]
    dt, ld, index = _need_product(rows, b, out, workspace, bias)
    xdt, xld = _matrix(x, rows, b.cols, b.device, "x")
    _check(_lib_mx4_linear(x.data_ptr(), xdt, xld, rows, b.ref, None if bias is None else bias.data_ptr(), int(relu),
                           out.data_ptr(), dt, ld, workspace.data_ptr(), workspace.nbytes,
                           _stream_of(stream, index, x, b.codes, b.scales, bias, out, workspace)), "iqlh_mx4_linear")


def iql_forward_values_mx4_workspace(h, batch):
    out = ctypes.c_size_t()
    _check(_lib_forward_mx4_ws(h, batch, ctypes.byref(out)), "iql_forward_values_mx4_workspace_bytes")
    return torch.empty(out.value, dtype=torch.uint8, device=torch.device("cuda", torch.cuda.current_device()))


def iql_forward_values_mx4(h, next_states, batch, out_v, workspace, rewards=None, dones=None, gamma=0.99,
                           out_target=None, states_ld=None, stream=None):
    """iql_forward_values with both hidden layers' operands in 4 bits.  next_states:
    [batch or more, S] with neighbouring columns, or of any shape with states_ld."""
    device = next_states.device
    index = _need_current(device)
    _need(next_states.dtype in (torch.float32, torch.bfloat16), "next_states must be float32 or bfloat16")
    _need(next_states.dim() > 0 and (next_states.shape[-1] <= 1 or next_states.stride(-1) == 1),
          "next_states must have neighbouring columns")
    if states_ld is None:
        _need(next_states.dim() == 2 and next_states.shape[0] >= batch, f"next_states must be {batch} rows or more")
    _need_f32(out_v, batch, device, "out_v")
    for t, what in ((rewards, "rewards"), (dones, "dones"), (out_target, "out_target")):
        if t is not None:
            _need_f32(t, batch, device, what)
    _need_aux(device, workspace, None)
    ld = states_ld if states_ld is not None else next_states.stride(0)
    _check(_lib_forward_mx4(h, _ptr(next_states), _DTYPES[next_states.dtype], ld, batch, _ptr(out_v), _ptr(rewards),
                            _ptr(dones), gamma, _ptr(out_target), _ptr(workspace),
                            workspace.numel() * workspace.element_size(),
                            _stream_of(stream, index, next_states, out_v, workspace, rewards, dones, out_target)),
           "iql_forward_values_mx4")


# ------------------------------------------------------------------- HER
def her_relabel(cfg, buf, source_idx, n, seed, d_step, out, stream=None):
    """cfg: HerConfig, buf: HerBuffer, out: HerOut (device addresses filled in)."""
    step = None if d_step is None else (d_step if isinstance(d_step, int) else d_step.data_ptr())
    _check(_lib_her_relabel(ctypes.byref(cfg), ctypes.byref(buf), _ptr(source_idx), n, seed,
                            None if step is None else ctypes.c_void_p(step), ctypes.byref(out),
                            _stream(stream)), "her_relabel")


def her_config(state_dim, goal_dim, strategy, goal_threshold=0.01, reward_hit=1.0, reward_miss=-0.01):
    c = HerConfig()
    c.state_dim, c.goal_dim, c.strategy = state_dim, goal_dim, strategy
    c.goal_threshold, c.reward_hit, c.reward_miss = goal_threshold, reward_hit, reward_miss
    return c


def her_buffer(states, next_states, actions, dones, episode_ends, buffer_size=None, rewards=None):
    """HerBuffer over device tensors.  The struct holds raw addresses, so it
    keeps references to the tensors: they stay allocated while it lives (a
    captured graph that replays a launch built from it needs that too)."""
    b = HerBuffer()
    b._keep = (states, next_states, actions, dones, episode_ends, rewards)
    b.states, b.next_states = states.data_ptr(), next_states.data_ptr()
    b.actions = actions.data_ptr() if actions is not None else None
    b.rewards = rewards.data_ptr() if rewards is not None else None
    b.dones = dones.data_ptr() if dones is not None else None
    b.episode_ends = episode_ends.data_ptr() if episode_ends is not None else None
    b.capacity = states.shape[0]
    b.buffer_size = states.shape[0] if buffer_size is None else buffer_size
    b.num_episodes = 0 if episode_ends is None else episode_ends.shape[0]
    return b


def her_out(states, states_dtype, states_ld, rewards, next_states=None, actions=None, dones=None,
            donor_idx=None, d_flags=None, is_weights=None):
    """HerOut; keeps references to the tensors it was given (see her_buffer).
    `states` and `is_weights` may be a tensor or a raw device address (a view
    into the merged batch)."""
    o = HerOut()
    o._keep = (states, rewards, next_states, actions, dones, donor_idx, d_flags, is_weights)
    o.states = states if isinstance(states, int) else states.data_ptr()
    o.states_dtype, o.states_ld = states_dtype, states_ld
    o.rewards = rewards.data_ptr()
    o.next_states = next_states.data_ptr() if next_states is not None else None
    o.actions = actions.data_ptr() if actions is not None else None
    o.dones = dones.data_ptr() if dones is not None else None
    o.donor_idx = donor_idx.data_ptr() if donor_idx is not None else None
    o.d_flags = d_flags if (d_flags is None or isinstance(d_flags, int)) else d_flags.data_ptr()
    o.is_weights = is_weights if (is_weights is None or isinstance(is_weights, int)) else is_weights.data_ptr()
    return o


# --------------------------------------------------------------- budget
def grad_budget_workspace_bytes(n, num_sources):
    out = ctypes.c_size_t()
    _check(_lib_ws_bytes(n, num_sources, ctypes.byref(out)), "grad_budget_workspace_bytes")
    return out.value


def make_adam(params, m, v, t, lr=3e-4, beta1=0.9, beta2=0.999, eps=1e-8, weight_decay=0.0,
              max_grad_norm=1.0, weight_clamp_max_abs=0.0, d_flags=None):
    """Adam state struct; keeps references to the tensors (see her_buffer)."""
    a = Adam()
    a._keep = (params, m, v, t, d_flags)
    a.params, a.m, a.v, a.t = params.data_ptr(), m.data_ptr(), v.data_ptr(), t.data_ptr()
    a.d_flags = None if d_flags is None else (d_flags if isinstance(d_flags, int) else d_flags.data_ptr())
    a.lr, a.beta1, a.beta2, a.eps = lr, beta1, beta2, eps
    a.weight_decay, a.max_grad_norm, a.weight_clamp_max_abs = weight_decay, max_grad_norm, weight_clamp_max_abs
    return a


def grad_budget_accumulate(grad_buf, sources, fractions, alphas, n, max_grad_norm, out_norms, adam,
                           workspace, stream=None):
    k = len(sources)
    srcs = (_p * k)(*[s.data_ptr() for s in sources])
    fr = (_f * k)(*fractions)
    al = (_f * k)(*alphas)
    _check(_lib_budget(_ptr(grad_buf), srcs, fr, al, k, n, max_grad_norm, _ptr(out_norms),
                       None if adam is None else ctypes.byref(adam), _ptr(workspace),
                       workspace.numel() * workspace.element_size(), _stream(stream)),
           "grad_budget_accumulate")


def grad_budget_accumulate_noalloc(grad_buf, sources, fractions, alphas, n, max_grad_norm, out_norms, adam,
                                   stream=None):
    """grad_budget_accumulate on the library's static device scratch (no workspace)."""
    k = len(sources)
    srcs = (_p * k)(*[s.data_ptr() for s in sources])
    fr = (_f * k)(*fractions)
    al = (_f * k)(*alphas)
    _check(_lib_budget_noalloc(_ptr(grad_buf), srcs, fr, al, k, n, max_grad_norm, _ptr(out_norms),
                               None if adam is None else ctypes.byref(adam), _stream(stream)),
           "grad_budget_accumulate_noalloc")


# ------------------------------------------------------------ whole step
def her_step(cfg, buf, source_idx, n, seed, out):
    """HerStep for iql_aux_step (the HER arguments of her_relabel minus d_step)."""
    st = HerStep()
    st._keep = (cfg, buf, out, source_idx)
    st.cfg, st.buf, st.out = ctypes.pointer(cfg), ctypes.pointer(buf), ctypes.pointer(out)
    st.source_idx = None if source_idx is None else source_idx.data_ptr()
    st.seed, st.n = seed, n
    return st


def budget_step(grad_buf, sources, fractions, alphas, n, max_grad_norm, out_norms, adam, workspace):
    """BudgetStep for iql_aux_step (the arguments of grad_budget_accumulate)."""
    k = len(sources)
    st = BudgetStep()
    st._keep = (grad_buf, tuple(sources), out_norms, adam, workspace)
    st.grad_buf = grad_buf.data_ptr()
    st.sources = (_p * k)(*[x.data_ptr() for x in sources])
    st.fractions = (_f * k)(*fractions)
    st.alphas = (_f * k)(*alphas)
    st.out_norms = None if out_norms is None else out_norms.data_ptr()
    if adam is not None:
        st.adam = ctypes.pointer(adam)
    st.workspace = workspace.data_ptr()
    st.workspace_bytes = workspace.numel() * workspace.element_size()
    st.n, st.num_sources, st.max_grad_norm = n, k, max_grad_norm
    return st


def iql_aux_step(h, her, states, q_taken, batch, q_all=None, num_actions=0, beta=0.0, out_pi=None, out_v=None,
                 out_loss=None, out_grad_norm=None, budget=None, stream=None):
    """HER + IQL step (+ AW policy) + budgeted accumulation in four launches."""
    _check(_lib_iql_aux_step(h, None if her is None else ctypes.byref(her), _ptr(states), _ptr(q_taken), batch,
                             _ptr(q_all), num_actions, beta, _ptr(out_pi), _ptr(out_v), _ptr(out_loss),
                             _ptr(out_grad_norm), None if budget is None else ctypes.byref(budget),
                             _stream(stream)), "iql_aux_step")


def iql_time_aux_step(h, her, states, q_taken, batch, q_all=None, num_actions=0, beta=0.0, out_pi=None,
                      out_v=None, out_loss=None, out_grad_norm=None, budget=None, reps=100, stream=None):
    """Runs `reps` whole steps with per-launch dispatch events; returns the mean
    duration (us) of launches [relabel+norms, forward/backward, reduce+SAXPY, Adam]."""
    out = (_f * 4)()
    _check(_lib_iql_time_aux_step(h, None if her is None else ctypes.byref(her), _ptr(states), _ptr(q_taken), batch,
                                  _ptr(q_all), num_actions, beta, _ptr(out_pi), _ptr(out_v), _ptr(out_loss),
                                  _ptr(out_grad_norm), None if budget is None else ctypes.byref(budget), reps, out,
                                  _stream(stream)), "iql_time_aux_step")
    return list(out)


PHASE_STAMPS = 8  # clock values per workgroup recorded by iql_aux_step_phase_stamps


def iql_aux_step_phase_stamps(h, her, states, q_taken, batch, q_all, num_actions, beta, out_pi, out_v, out_loss,
                              out_grad_norm, budget, stamps, stream=None):
    """iql_aux_step with the forward/backward kernel's phase ends recorded:
    `stamps` is a device int64 tensor of groups * ceil(batch / 128) *
    PHASE_STAMPS elements (100 MHz clock values, tile order)."""
    _check(_lib_iql_aux_step_phase_stamps(h, None if her is None else ctypes.byref(her), _ptr(states),
                                          _ptr(q_taken), batch, _ptr(q_all), num_actions, beta, _ptr(out_pi),
                                          _ptr(out_v), _ptr(out_loss), _ptr(out_grad_norm),
                                          None if budget is None else ctypes.byref(budget), _ptr(stamps),
                                          stamps.numel(), _stream(stream)), "iql_aux_step_phase_stamps")


class IqlTrainer:
    """Owns an iql_handle; methods forward to the C entry points."""

    def __init__(self, cfg, init_params_host):
        self.cfg = cfg
        self.h = iql_create(cfg, init_params_host)
        self.n_params = iql_config_num_params(cfg)

    def forward_values(self, next_states, batch, out_v, rewards=None, dones=None, gamma=0.99, out_target=None,
                       states_ld=None, stream=None):
        iql_forward_values(self.h, next_states, batch, out_v, rewards, dones, gamma, out_target, states_ld, stream)

    def forward_values_mx4_workspace(self, batch):
        return iql_forward_values_mx4_workspace(self.h, batch)

    def forward_values_mx4(self, next_states, batch, out_v, workspace, rewards=None, dones=None, gamma=0.99,
                           out_target=None, states_ld=None, stream=None):
        S, groups = self.cfg.state_dim, self.cfg.num_groups
        _need(next_states.dim() != 2 or next_states.shape[1] >= S, f"next_states must have {S} columns or more")
        for t, what in ((out_v, "out_v"), (out_target, "out_target")):
            if t is not None:
                _need_f32(t, groups * batch, next_states.device, what)
        iql_forward_values_mx4(self.h, next_states, batch, out_v, workspace, rewards, dones, gamma, out_target,
                               states_ld, stream)

    def target_ema_update(self, tau, stream=None):
        iql_target_ema_update(self.h, tau, stream)

    def set_target_ema(self, tau):
        iql_set_target_ema(self.h, tau)

    def get_target(self, group, params, stream=None):
        iql_get_target(self.h, group, params, stream)

    def set_target(self, group, params, stream=None):
        iql_set_target(self.h, group, params, stream)

    def partial_layout(self, batch):
        return iql_partial_layout(self.h, batch)

    def train_step(self, states, q_taken, batch, out_v=None, out_loss=None, out_grad_norm=None, stream=None):
        iql_train_step(self.h, states, q_taken, batch, out_v, out_loss, out_grad_norm, stream)

    def train_step_aw(self, states, q_taken, batch, q_all, num_actions, beta, out_pi, out_v, out_loss=None,
                      out_grad_norm=None, stream=None):
        iql_train_step_aw(self.h, states, q_taken, batch, q_all, num_actions, beta, out_pi, out_v, out_loss,
                          out_grad_norm, stream)

    def aux_step(self, her, states, q_taken, batch, q_all=None, num_actions=0, beta=0.0, out_pi=None, out_v=None,
                 out_loss=None, out_grad_norm=None, budget=None, stream=None):
        iql_aux_step(self.h, her, states, q_taken, batch, q_all, num_actions, beta, out_pi, out_v, out_loss,
                     out_grad_norm, budget, stream)

    def time_aux_step(self, her, states, q_taken, batch, q_all=None, num_actions=0, beta=0.0, out_pi=None,
                      out_v=None, out_loss=None, out_grad_norm=None, budget=None, reps=100, stream=None):
        return iql_time_aux_step(self.h, her, states, q_taken, batch, q_all, num_actions, beta, out_pi, out_v,
                                 out_loss, out_grad_norm, budget, reps, stream)

    def aux_step_phase_stamps(self, her, states, q_taken, batch, q_all, num_actions, beta, out_pi, out_v, out_loss,
                              out_grad_norm, budget, stamps, stream=None):
        iql_aux_step_phase_stamps(self.h, her, states, q_taken, batch, q_all, num_actions, beta, out_pi, out_v,
                                  out_loss, out_grad_norm, budget, stamps, stream)

    def compute_gradients(self, states, q_taken, batch, out_v=None, stream=None):
        iql_compute_gradients(self.h, states, q_taken, batch, out_v, stream)

    def apply_gradients(self, batch, out_loss=None, out_grad_norm=None, stream=None):
        iql_apply_gradients(self.h, batch, out_loss, out_grad_norm, stream)

    def get_state(self, group, params=None, m=None, v=None, t=None, stream=None):
        iql_get_state(self.h, group, params, m, v, t, stream)

    def set_state(self, group, params, m, v, t, stream=None):
        iql_set_state(self.h, group, params, m, v, t, stream)

    @property
    def step_counter(self):
        return iql_step_counter(self.h)

    @property
    def flags(self):
        return iql_flags(self.h)

    def status(self):
        return iql_status(self.h)

    def close(self):
        if self.h:
            iql_destroy(self.h)
            self.h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass
