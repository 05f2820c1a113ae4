"""Python binding of librollout.so: fused PPO experience collection on MI355X.

Argument marshalling only.  Every step of the collection runs in the HIP
kernels behind the C ABI of include/rollout.h; PyTorch supplies device
memory and the stream.  There is no CPU path: if the library is missing or
fails to load, importing the functions raises.

The functions carry the C names:
    rollout_config_default, rollout_create, rollout_set_weights,
    rollout_collect, gae_scan, gae_scan_noalloc, rollout_destroy,
    rollout_last_error
    (include/rollout.h), dqn_config_default, dqn_create,
    dqn_set_weights, dqn_set_epsilon, dqn_collect, dqn_destroy
    (include/dqn.h), and
    per_create, per_sample, per_gather, per_update, per_destroy
    (include/per.h).
The operators of a policy with memory (include/policy.h) are `embed`,
`recurrence`, `recurrence_step` and `shape_logits` (policy.py); all but the
step take part in torch's autograd.
There are also helpers: `alloc_outputs`, `alloc_dqn_outputs` and the `Collector` and
`DqnCollector` and `PerSampler` convenience classes.
"""
from __future__ import annotations

import ctypes as C
import os

PKG_DIR = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(PKG_DIR, "librollout.so")

ROLLOUT_OK, ROLLOUT_EINVAL, ROLLOUT_ENOMEM, ROLLOUT_EHIP, ROLLOUT_ENOTIMPL = 0, -1, -2, -3, -4
ROLLOUT_FP32, ROLLOUT_BF16 = 0, 1
STATE_DIM, N_ACTIONS, N_FEATURES = 54, 45, 51
STAMP_WORDS = 16  # per wave, rollout_phase_cycles
STAMP_PHASES = ("state assembly and stores", "state barrier", "first layer", "barrier",
                "second layer", "barrier", "third layer", "barrier", "draw",
                "environment step", "stores and reset")
EXPORTED = ("rollout_config_default", "rollout_create", "rollout_set_weights", "rollout_collect",
            "rollout_phase_cycles",
            "gae_scan", "gae_scan_noalloc", "rollout_destroy", "rollout_last_error",
            "dqn_config_default", "dqn_create", "dqn_set_weights", "dqn_set_epsilon",
            "dqn_collect", "dqn_destroy",
            "per_create", "per_sample", "per_gather", "per_update", "per_destroy")


class RolloutConfig(C.Structure):
    _fields_ = [
        ("n_episodes", C.c_int32), ("n_steps", C.c_int32),
        ("n_features", C.c_int32), ("state_dim", C.c_int32), ("n_actions", C.c_int32),
        ("actor_dims", C.c_int32 * 4), ("critic_dims", C.c_int32 * 7), ("cur_dims", C.c_int32 * 3),
        ("precision", C.c_int32),
        ("gamma", C.c_float), ("lam", C.c_float),
        ("profit_take", C.c_float), ("stop_loss", C.c_float), ("max_hold", C.c_int32),
        ("div_window", C.c_int32), ("div_threshold", C.c_float), ("div_penalty", C.c_float),
        ("curiosity_coef", C.c_float), ("risk_coef", C.c_float), ("spread", C.c_float),
        ("barrier_scale", C.c_float),
        ("exposure", C.c_float * 5), ("cost", C.c_float * 3), ("urgency_mult", C.c_float),
        ("recycle", C.c_int32), ("overlap", C.c_int32),
    ]


class RolloutOutputs(C.Structure):
    _fields_ = [(n, C.c_void_p) for n in (
        "states", "actions", "log_probs", "values", "rewards", "dones", "barrier",
        "advantages", "returns", "logits", "counters", "phase_events")]


class DqnConfig(C.Structure):
    _fields_ = [
        ("n_episodes", C.c_int32), ("n_steps", C.c_int32),
        ("n_features", C.c_int32), ("state_dim", C.c_int32), ("n_actions", C.c_int32),
        ("trunk_dims", C.c_int32 * 3), ("value_dims", C.c_int32 * 3),
        ("advantage_dims", C.c_int32 * 3), ("cur_dims", C.c_int32 * 3),
        ("epsilon", C.c_float), ("gamma", C.c_float), ("priority_alpha", C.c_float),
        ("profit_take", C.c_float), ("stop_loss", C.c_float), ("max_hold", C.c_int32),
        ("div_window", C.c_int32), ("div_threshold", C.c_float), ("div_penalty", C.c_float),
        ("curiosity_coef", C.c_float), ("risk_coef", C.c_float), ("spread", C.c_float),
        ("barrier_scale", C.c_float),
        ("exposure", C.c_float * 5), ("cost", C.c_float * 3), ("urgency_mult", C.c_float),
        ("recycle", C.c_int32),
    ]


class DqnOutputs(C.Structure):
    _fields_ = [(n, C.c_void_p) for n in (
        "states", "next_states", "q_values", "actions", "explored", "q_taken", "q_next_max",
        "rewards", "dones", "barrier", "td", "priorities", "counters", "phase_events")]


class RolloutError(RuntimeError):
    def __init__(self, code: int, msg: str):
        super().__init__(f"[{code}] {msg}")
        self.code = code


_lib = None


def load_library(path: str = LIB_PATH):
    """Load librollout.so (raises if it is missing: there is no fallback)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(path):
        raise ImportError(f"{path} is not built; run __graft_entry__.build() "
                          "(or python rl_experience_collection_amd/build.py)")
    # torch's HIP runtime has the same soname as the system one: load it
    # first, so this library binds to the runtime torch's tensors and streams
    # live in (loaded first, it would bind torch to the system copy instead)
    try:
        import torch  # noqa: F401
    except ImportError:
        pass
    L = C.CDLL(path)
    vp, i32, i64 = C.c_void_p, C.c_int32, C.c_int64
    L.rollout_config_default.argtypes = [C.POINTER(RolloutConfig), i32, i32]
    L.rollout_create.argtypes = [C.POINTER(RolloutConfig), C.POINTER(vp), C.POINTER(vp),
                                 C.POINTER(vp), vp, vp, i64, vp, C.POINTER(vp)]
    L.rollout_set_weights.argtypes = [vp, C.POINTER(vp), C.POINTER(vp), C.POINTER(vp), vp]
    L.rollout_collect.argtypes = [vp, vp, C.c_uint64, C.POINTER(RolloutOutputs), vp]
    L.rollout_phase_cycles.argtypes = [vp, i32, vp, i64, C.POINTER(i64)]
    L.gae_scan.argtypes = [vp, vp, vp, vp, i32, i32, C.c_float, C.c_float, vp, vp, vp]
    L.gae_scan_noalloc.argtypes = L.gae_scan.argtypes
    L.rollout_destroy.argtypes = [vp]
    L.rollout_destroy.restype = None
    L.rollout_last_error.argtypes = []
    L.rollout_last_error.restype = C.c_char_p
    L.dqn_config_default.argtypes = [C.POINTER(DqnConfig), i32, i32]
    L.dqn_create.argtypes = [C.POINTER(DqnConfig), C.POINTER(vp), C.POINTER(vp), C.POINTER(vp),
                             vp, vp, i64, vp, C.POINTER(vp)]
    L.dqn_set_weights.argtypes = [vp, C.POINTER(vp), C.POINTER(vp), C.POINTER(vp), vp]
    L.dqn_set_epsilon.argtypes = [vp, C.c_float]
    L.dqn_collect.argtypes = [vp, vp, C.c_uint64, C.POINTER(DqnOutputs), vp]
    L.dqn_destroy.argtypes = [vp]
    L.dqn_destroy.restype = None
    f32 = C.c_float
    L.per_create.argtypes = [i64, i32, C.POINTER(vp)]
    L.per_sample.argtypes = [vp, vp, i64, i32, C.c_uint64, f32, vp, vp, vp]
    L.per_gather.argtypes = [vp, i32, i64, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp]
    L.per_update.argtypes = [vp, i64, vp, vp, i32, f32, f32, f32, vp]
    L.per_destroy.argtypes = [vp]
    L.per_destroy.restype = None
    for name in ("rollout_config_default", "rollout_create", "rollout_set_weights",
                 "rollout_collect", "rollout_phase_cycles", "gae_scan", "gae_scan_noalloc", "dqn_config_default",
                 "dqn_create",
                 "dqn_set_weights", "dqn_set_epsilon", "dqn_collect", "per_create", "per_sample", "per_gather",
                 "per_update"):
        getattr(L, name).restype = C.c_int
    try:
        import torch  # noqa: F401
    except ImportError:
        pass
    else:
        from . import policy
        policy.declare(L)
    _lib = L
    return L


def rollout_last_error() -> str:
    return load_library().rollout_last_error().decode()


def _check(rc: int):
    if rc != ROLLOUT_OK:
        raise RolloutError(rc, rollout_last_error())


# ----------------------------------------------------------------- marshalling
def _stream(stream):
    import torch
    if stream is None:
        return C.c_void_p(torch.cuda.current_stream().cuda_stream)
    if isinstance(stream, int):
        return C.c_void_p(stream)
    return C.c_void_p(stream.cuda_stream)


def _dev_ptr(t, dtype, shape=None, name="tensor"):
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError(f"{name} must be a device tensor")
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    return C.c_void_p(t.data_ptr())


def _ptr_array(tensors, shapes, name):
    import torch
    if len(tensors) != len(shapes):
        raise ValueError(f"{name}: expected {len(shapes)} tensors, got {len(tensors)}")
    arr = (C.c_void_p * len(tensors))()
    for i, (t, s) in enumerate(zip(tensors, shapes)):
        arr[i] = _dev_ptr(t, torch.float32, s, f"{name}[{i}]").value
    return arr


ACTOR_SHAPES = [(128, 54), (128,), (64, 128), (64,), (45, 64), (45,)]
CRITIC_SHAPES = [(512, 54), (512,), (384, 512), (384,), (256, 384), (256,), (128, 256), (128,),
                 (64, 128), (64,), (1, 64), (1,)]
CURIOSITY_SHAPES = [(128, 99), (128,), (51, 128), (51,)]


def rollout_config_default(n_episodes: int, n_steps: int, settings: dict | None = None,
                           precision: int = ROLLOUT_FP32) -> RolloutConfig:
    cfg = RolloutConfig()
    _check(load_library().rollout_config_default(C.byref(cfg), n_episodes, n_steps))
    cfg.precision = precision
    for k, v in (settings or {}).items():
        if k in ("exposure", "cost"):
            setattr(cfg, k, (C.c_float * len(v))(*v))
        elif k == "lambda":
            cfg.lam = v
        else:
            setattr(cfg, k, v)
    return cfg


def rollout_create(cfg: RolloutConfig, actor, critic, curiosity, features, prices, stream=None):
    """Returns an opaque handle (int).  The market tensors are borrowed."""
    import torch
    a = _ptr_array(actor, ACTOR_SHAPES, "actor")
    c = _ptr_array(critic, CRITIC_SHAPES, "critic")
    u = _ptr_array(curiosity, CURIOSITY_SHAPES, "curiosity")
    if features.dim() != 2 or features.shape[1] != N_FEATURES:
        raise ValueError("features must be [n_bars, 51]")
    f = _dev_ptr(features, torch.float32, name="features")
    p = _dev_ptr(prices, torch.float32, (features.shape[0],), "prices")
    h = C.c_void_p()
    _check(load_library().rollout_create(C.byref(cfg), a, c, u, f, p, features.shape[0],
                                         _stream(stream), C.byref(h)))
    return h.value


def rollout_set_weights(handle: int, actor, critic, curiosity, stream=None):
    a = _ptr_array(actor, ACTOR_SHAPES, "actor")
    c = _ptr_array(critic, CRITIC_SHAPES, "critic")
    u = _ptr_array(curiosity, CURIOSITY_SHAPES, "curiosity")
    _check(load_library().rollout_set_weights(C.c_void_p(handle), a, c, u, _stream(stream)))


def alloc_outputs(N: int, L: int, device="cuda", logits: bool = False, counters: bool = True):
    import torch
    f32 = dict(dtype=torch.float32, device=device)
    out = dict(
        states=torch.empty((L, N, STATE_DIM), **f32),
        actions=torch.empty((L, N), dtype=torch.int32, device=device),
        log_probs=torch.empty((L, N), **f32),
        values=torch.empty((L, N), **f32),
        rewards=torch.empty((L, N), **f32),
        dones=torch.empty((L, N), dtype=torch.uint8, device=device),
        barrier=torch.empty((L, N), dtype=torch.uint8, device=device),
        advantages=torch.empty((L, N), **f32),
        returns=torch.empty((L, N), **f32),
        logits=torch.empty((L, N, N_ACTIONS), **f32) if logits else None,
        counters=torch.zeros(3, dtype=torch.int32, device=device) if counters else None,
    )
    return out


def rollout_collect(handle: int, episode_starts, seed: int, outputs: dict, stream=None,
                    phase_events=None):
    """phase_events: None or a sequence of 4 hipEvent_t handles (ints)."""
    import torch
    L, N = outputs["actions"].shape
    o = RolloutOutputs()
    o.states = _dev_ptr(outputs["states"], torch.float32, (L, N, STATE_DIM), "states")
    o.actions = _dev_ptr(outputs["actions"], torch.int32, (L, N), "actions")
    o.log_probs = _dev_ptr(outputs["log_probs"], torch.float32, (L, N), "log_probs")
    o.values = _dev_ptr(outputs["values"], torch.float32, (L, N), "values")
    o.rewards = _dev_ptr(outputs["rewards"], torch.float32, (L, N), "rewards")
    o.dones = _dev_ptr(outputs["dones"], torch.uint8, (L, N), "dones")
    o.barrier = _dev_ptr(outputs["barrier"], torch.uint8, (L, N), "barrier")
    o.advantages = _dev_ptr(outputs["advantages"], torch.float32, (L, N), "advantages")
    o.returns = _dev_ptr(outputs["returns"], torch.float32, (L, N), "returns")
    o.logits = _dev_ptr(outputs.get("logits"), torch.float32, (L, N, N_ACTIONS), "logits")
    o.counters = _dev_ptr(outputs.get("counters"), torch.int32, (3,), "counters")
    ev = None
    if phase_events is not None:
        if len(phase_events) != 4:
            raise ValueError("phase_events must hold 4 event handles")
        ev = (C.c_void_p * 4)(*phase_events)
        o.phase_events = C.cast(ev, C.c_void_p)
    s = _dev_ptr(episode_starts, torch.int32, (N,), "episode_starts")
    _check(load_library().rollout_collect(C.c_void_p(handle), s, C.c_uint64(seed), C.byref(o),
                                          _stream(stream)))


def gae_scan(rewards, values, dones, last_values, gamma: float, lam: float, advantages, returns,
             stream=None, noalloc: bool = False):
    """noalloc=True calls gae_scan_noalloc (no device allocation; its scratch
    is a fixed array of the library)."""
    import torch
    L, N = rewards.shape
    lib = load_library()
    fn = lib.gae_scan_noalloc if noalloc else lib.gae_scan
    _check(fn(
        _dev_ptr(rewards, torch.float32, (L, N), "rewards"),
        _dev_ptr(values, torch.float32, (L, N), "values"),
        _dev_ptr(dones, torch.uint8, (L, N), "dones"),
        _dev_ptr(last_values, torch.float32, (N,), "last_values"),
        L, N, gamma, lam,
        _dev_ptr(advantages, torch.float32, (L, N), "advantages"),
        _dev_ptr(returns, torch.float32, (L, N), "returns"),
        _stream(stream)))


def rollout_destroy(handle: int):
    if handle:
        load_library().rollout_destroy(C.c_void_p(handle))


class HipEvents:
    """Timing events created through the HIP runtime (for phase_events)."""

    def __init__(self, n: int):
        self._hip = C.CDLL("libamdhip64.so")
        self._hip.hipEventCreate.argtypes = [C.POINTER(C.c_void_p)]
        self._hip.hipEventElapsedTime.argtypes = [C.POINTER(C.c_float), C.c_void_p, C.c_void_p]
        self._hip.hipEventDestroy.argtypes = [C.c_void_p]
        self._hip.hipEventRecord.argtypes = [C.c_void_p, C.c_void_p]
        self.handles = []
        for _ in range(n):
            e = C.c_void_p()
            if self._hip.hipEventCreate(C.byref(e)) != 0:
                raise RuntimeError("hipEventCreate failed")
            self.handles.append(e.value)

    def record(self, i: int, stream=None):
        if self._hip.hipEventRecord(C.c_void_p(self.handles[i]), _stream(stream)) != 0:
            raise RuntimeError("hipEventRecord failed")

    def elapsed_ms(self, i: int, j: int) -> float:
        ms = C.c_float()
        if self._hip.hipEventElapsedTime(C.byref(ms), C.c_void_p(self.handles[i]),
                                         C.c_void_p(self.handles[j])) != 0:
            raise RuntimeError("hipEventElapsedTime failed")
        return ms.value

    def close(self):
        for h in self.handles:
            self._hip.hipEventDestroy(C.c_void_p(h))
        self.handles = []


class Collector:
    """Owns one handle; weights as lists of [out, in] fp32 device tensors."""

    def __init__(self, n_episodes: int, n_steps: int, weights: dict, features, prices,
                 settings: dict | None = None, precision: int = ROLLOUT_FP32, stream=None):
        self.N, self.L = n_episodes, n_steps
        self.cfg = rollout_config_default(n_episodes, n_steps, settings, precision)
        self.features, self.prices = features, prices  # borrowed by the library
        self.handle = rollout_create(self.cfg, weights["actor"], weights["critic"],
                                     weights["curiosity"], features, prices, stream)

    def set_weights(self, weights: dict, stream=None):
        rollout_set_weights(self.handle, weights["actor"], weights["critic"],
                            weights["curiosity"], stream)

    def collect(self, episode_starts, seed: int, outputs: dict | None = None, logits=False,
                stream=None, phase_events=None) -> dict:
        if outputs is None:
            outputs = alloc_outputs(self.N, self.L, episode_starts.device, logits=logits)
        rollout_collect(self.handle, episode_starts, seed, outputs, stream, phase_events)
        return outputs

    def phase_cycles(self, enable: bool):
        """rollout_phase_cycles: switch the instrumented step kernel on or
        off for later collections and return the per-wave cycle totals
        gathered since the last call, shape [waves, STAMP_WORDS] (uint64)."""
        import numpy as np
        waves = 4 * -(-self.N // 16)
        out = np.zeros((waves, STAMP_WORDS), np.uint64)
        n = C.c_int64()
        _check(load_library().rollout_phase_cycles(
            C.c_void_p(self.handle), int(bool(enable)), out.ctypes.data_as(C.c_void_p),
            out.size, C.byref(n)))
        return out

    def close(self):
        if self.handle:
            rollout_destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


# --------------------------------------------------------------------------- DQN
Q_NET_SHAPES = [(256, 54), (256,), (128, 256), (128,), (64, 128), (64,), (1, 64), (1,),
                (64, 128), (64,), (45, 64), (45,)]


def dqn_config_default(n_episodes: int, n_steps: int, settings: dict | None = None,
                       dqn: dict | None = None) -> DqnConfig:
    """settings: environment scalars (as for rollout_config_default); dqn:
    {'epsilon', 'gamma', 'alpha'}."""
    cfg = DqnConfig()
    _check(load_library().dqn_config_default(C.byref(cfg), n_episodes, n_steps))
    for k, v in (settings or {}).items():
        if k in ("gamma", "lam", "lambda"):
            continue  # GAE settings of the PPO collection
        if k in ("exposure", "cost"):
            setattr(cfg, k, (C.c_float * len(v))(*v))
        else:
            setattr(cfg, k, v)
    for k, v in (dqn or {}).items():
        setattr(cfg, "priority_alpha" if k == "alpha" else k, v)
    return cfg


def _nullable_array(tensors, shapes, name):
    return None if tensors is None else _ptr_array(tensors, shapes, name)


def dqn_create(cfg: DqnConfig, online, target, curiosity, features, prices, stream=None):
    """Returns an opaque handle (int).  The market tensors are borrowed."""
    import torch
    o = _ptr_array(online, Q_NET_SHAPES, "online")
    t = _ptr_array(target, Q_NET_SHAPES, "target")
    u = _ptr_array(curiosity, CURIOSITY_SHAPES, "curiosity")
    if features.dim() != 2 or features.shape[1] != N_FEATURES:
        raise ValueError("features must be [n_bars, 51]")
    f = _dev_ptr(features, torch.float32, name="features")
    p = _dev_ptr(prices, torch.float32, (features.shape[0],), "prices")
    h = C.c_void_p()
    _check(load_library().dqn_create(C.byref(cfg), o, t, u, f, p, features.shape[0],
                                     _stream(stream), C.byref(h)))
    return h.value


def dqn_set_weights(handle: int, online=None, target=None, curiosity=None, stream=None):
    """None keeps that network."""
    _check(load_library().dqn_set_weights(
        C.c_void_p(handle), _nullable_array(online, Q_NET_SHAPES, "online"),
        _nullable_array(target, Q_NET_SHAPES, "target"),
        _nullable_array(curiosity, CURIOSITY_SHAPES, "curiosity"), _stream(stream)))


def dqn_set_epsilon(handle: int, epsilon: float):
    """Exploration probability of the collections enqueued after this call."""
    _check(load_library().dqn_set_epsilon(C.c_void_p(handle), float(epsilon)))


def alloc_dqn_outputs(N: int, L: int, device="cuda", next_states: bool = True,
                      q_values: bool = False, explored: bool = True, counters: bool = True):
    import torch
    f32 = dict(dtype=torch.float32, device=device)
    u8 = dict(dtype=torch.uint8, device=device)
    return dict(
        states=torch.empty((L, N, STATE_DIM), **f32),
        next_states=torch.empty((L, N, STATE_DIM), **f32) if next_states else None,
        q_values=torch.empty((L, N, N_ACTIONS), **f32) if q_values else None,
        actions=torch.empty((L, N), dtype=torch.int32, device=device),
        explored=torch.empty((L, N), **u8) if explored else None,
        q_taken=torch.empty((L, N), **f32),
        q_next_max=torch.empty((L, N), **f32),
        rewards=torch.empty((L, N), **f32),
        dones=torch.empty((L, N), **u8),
        barrier=torch.empty((L, N), **u8),
        td=torch.empty((L, N), **f32),
        priorities=torch.empty((L, N), **f32),
        counters=torch.zeros(2, dtype=torch.int32, device=device) if counters else None,
    )


def dqn_collect(handle: int, episode_starts, seed: int, outputs: dict, stream=None,
                phase_events=None):
    """phase_events: None or a sequence of 2 hipEvent_t handles (ints)."""
    import torch
    L, N = outputs["actions"].shape
    o = DqnOutputs()
    o.states = _dev_ptr(outputs["states"], torch.float32, (L, N, STATE_DIM), "states")
    o.next_states = _dev_ptr(outputs.get("next_states"), torch.float32, (L, N, STATE_DIM),
                             "next_states")
    o.q_values = _dev_ptr(outputs.get("q_values"), torch.float32, (L, N, N_ACTIONS), "q_values")
    o.actions = _dev_ptr(outputs["actions"], torch.int32, (L, N), "actions")
    o.explored = _dev_ptr(outputs.get("explored"), torch.uint8, (L, N), "explored")
    for k in ("q_taken", "q_next_max", "rewards", "td", "priorities"):
        setattr(o, k, _dev_ptr(outputs[k], torch.float32, (L, N), k))
    o.dones = _dev_ptr(outputs["dones"], torch.uint8, (L, N), "dones")
    o.barrier = _dev_ptr(outputs["barrier"], torch.uint8, (L, N), "barrier")
    o.counters = _dev_ptr(outputs.get("counters"), torch.int32, (2,), "counters")
    ev = None
    if phase_events is not None:
        if len(phase_events) != 2:
            raise ValueError("phase_events must hold 2 event handles")
        ev = (C.c_void_p * 2)(*phase_events)
        o.phase_events = C.cast(ev, C.c_void_p)
    s = _dev_ptr(episode_starts, torch.int32, (N,), "episode_starts")
    _check(load_library().dqn_collect(C.c_void_p(handle), s, C.c_uint64(seed), C.byref(o),
                                      _stream(stream)))


def dqn_destroy(handle: int):
    if handle:
        load_library().dqn_destroy(C.c_void_p(handle))


class DqnCollector:
    """Owns one DQN handle; weights as lists of [out, in] fp32 device tensors."""

    def __init__(self, n_episodes: int, n_steps: int, weights: dict, features, prices,
                 settings: dict | None = None, dqn: dict | None = None, stream=None):
        self.N, self.L = n_episodes, n_steps
        self.cfg = dqn_config_default(n_episodes, n_steps, settings, dqn)
        self.features, self.prices = features, prices  # borrowed by the library
        self.handle = dqn_create(self.cfg, weights["online"], weights["target"],
                                 weights["curiosity"], features, prices, stream)

    def set_weights(self, online=None, target=None, curiosity=None, stream=None):
        dqn_set_weights(self.handle, online, target, curiosity, stream)

    def set_epsilon(self, epsilon: float):
        dqn_set_epsilon(self.handle, epsilon)

    def collect(self, episode_starts, seed: int, outputs: dict | None = None, q_values=False,
                stream=None, phase_events=None) -> dict:
        if outputs is None:
            outputs = alloc_dqn_outputs(self.N, self.L, episode_starts.device, q_values=q_values)
        dqn_collect(self.handle, episode_starts, seed, outputs, stream, phase_events)
        return outputs

    def close(self):
        if self.handle:
            dqn_destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


# ------------------------------------------------------------- prioritized replay
def per_create(capacity: int, max_batch: int) -> int:
    h = C.c_void_p()
    _check(load_library().per_create(capacity, max_batch, C.byref(h)))
    return h.value


def per_sample(handle: int, priorities, batch: int, seed: int, beta: float, indices, weights,
               stream=None):
    import torch
    n = priorities.numel()
    _check(load_library().per_sample(
        C.c_void_p(handle), _dev_ptr(priorities, torch.float32, (n,), "priorities"), n, batch,
        C.c_uint64(seed), beta, _dev_ptr(indices, torch.int32, (batch,), "indices"),
        _dev_ptr(weights, torch.float32, (batch,), "weights"), _stream(stream)))


def per_gather(indices, n: int, states=None, next_states=None, actions=None, rewards=None,
               dones=None, out: dict | None = None, stream=None) -> dict:
    """Sources are flat [n(, 54)] views (a [L][N] collection output reshaped);
    returns the batch arrays (allocated when `out` is None)."""
    import torch
    B = indices.numel()
    dev = indices.device
    src = dict(states=states, next_states=next_states, actions=actions, rewards=rewards, dones=dones)
    if out is None:
        mk = dict(states=lambda: torch.empty((B, STATE_DIM), dtype=torch.float32, device=dev),
                  next_states=lambda: torch.empty((B, STATE_DIM), dtype=torch.float32, device=dev),
                  actions=lambda: torch.empty(B, dtype=torch.int32, device=dev),
                  rewards=lambda: torch.empty(B, dtype=torch.float32, device=dev),
                  dones=lambda: torch.empty(B, dtype=torch.uint8, device=dev))
        out = {k: (mk[k]() if v is not None else None) for k, v in src.items()}
    types = dict(states=torch.float32, next_states=torch.float32, actions=torch.int32,
                 rewards=torch.float32, dones=torch.uint8)
    shp = lambda k, m: (m, STATE_DIM) if k in ("states", "next_states") else (m,)
    ps = [_dev_ptr(src[k], types[k], shp(k, n), k) for k in src]
    po = [_dev_ptr(out[k], types[k], shp(k, B), "out_" + k) if out.get(k) is not None else None
          for k in src]
    _check(load_library().per_gather(_dev_ptr(indices, torch.int32, (B,), "indices"), B, n, *ps,
                                     *po, _stream(stream)))
    return out


def per_update(priorities, indices, td, alpha: float, epsilon: float, max_priority: float,
               stream=None):
    import torch
    n, B = priorities.numel(), indices.numel()
    _check(load_library().per_update(
        _dev_ptr(priorities, torch.float32, (n,), "priorities"), n,
        _dev_ptr(indices, torch.int32, (B,), "indices"), _dev_ptr(td, torch.float32, (B,), "td"),
        B, alpha, epsilon, max_priority, _stream(stream)))


def per_destroy(handle: int):
    if handle:
        load_library().per_destroy(C.c_void_p(handle))


class PerSampler:
    """Owns one sampler handle."""

    def __init__(self, capacity: int, max_batch: int):
        self.capacity, self.max_batch = capacity, max_batch
        self.handle = per_create(capacity, max_batch)

    def sample(self, priorities, batch: int, seed: int, beta: float, stream=None):
        import torch
        idx = torch.empty(batch, dtype=torch.int32, device=priorities.device)
        w = torch.empty(batch, dtype=torch.float32, device=priorities.device)
        per_sample(self.handle, priorities, batch, seed, beta, idx, w, stream)
        return idx, w

    def close(self):
        if self.handle:
            per_destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


# ---------------------------------------------------------- policies with memory
_POLICY = ("embed", "recurrence", "recurrence_step", "shape_logits")


def __getattr__(name):
    # policy.py imports torch, which a caller of the C names may lack
    if name in _POLICY:
        from . import policy
        for n in _POLICY:
            globals()[n] = getattr(policy, n)
        return globals()[name]
    raise AttributeError(f"module {__name__!r} has no attribute {name!r}")
