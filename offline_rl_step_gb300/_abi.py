"""ctypes declarations of the C ABI in include/ofrl.h (argument marshalling only)."""
import ctypes as C
import os

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libofrl.so")

OK, EINVAL, EUNSUPPORTED, ECUDA, ETIMEOUT = 0, -1, -2, -3, -4
HER_FINAL, HER_FUTURE, HER_RANDOM, HER_EPISODE = 0, 1, 2, 3
PREC_FP32, PREC_BF16 = 0, 1
STAT_NONFINITE_GRAD, STAT_BAD_ACTION, STAT_BAD_INDEX, STAT_TIMEOUT, STAT_SANITIZED, STAT_WORDS = 0, 1, 2, 3, 4, 8

vp = C.c_void_p


class Replay(C.Structure):
    _fields_ = [("states", vp), ("next_states", vp), ("actions", vp), ("rewards", vp), ("dones", vp),
                ("episode_ends", vp), ("capacity", C.c_int64), ("num_episodes", C.c_int32),
                ("state_dim", C.c_int32), ("state_stride", C.c_int32), ("goal_dim", C.c_int32)]


class HerCfg(C.Structure):
    _fields_ = [("batch", C.c_int32), ("her_count", C.c_int32), ("strategy", C.c_int32),
                ("goal_threshold", C.c_float), ("seed", C.c_uint64)]


class Batch(C.Structure):
    _fields_ = [("states", vp), ("next_states", vp), ("actions", vp), ("rewards", vp), ("dones", vp),
                ("src_idx", vp), ("donor_idx", vp), ("stride", C.c_int32)]


class VShape(C.Structure):
    _fields_ = [("state_dim", C.c_int32), ("hidden", C.c_int32), ("num_actions", C.c_int32),
                ("prec", C.c_int32)]


class VNet(C.Structure):
    _fields_ = [("params", vp), ("m", vp), ("v", vp), ("t", C.c_int32), ("tau", C.c_float), ("target", vp),
                ("polyak", C.c_float)]


class Opt(C.Structure):
    _fields_ = [("lr", C.c_float), ("beta1", C.c_float), ("beta2", C.c_float), ("eps", C.c_float),
                ("weight_decay", C.c_float), ("max_grad_norm", C.c_float), ("beta", C.c_float),
                ("budget", C.c_float * 4), ("alpha", C.c_float * 4), ("weight_clamp_max_abs", C.c_float),
                ("sanitize_sources", C.c_int32)]


DTYPE_F32, DTYPE_BF16 = 0, 1


class DeltaShape(C.Structure):
    _fields_ = [("k_heads", C.c_int32), ("v_heads", C.c_int32), ("k_dim", C.c_int32), ("v_dim", C.c_int32),
                ("dtype", C.c_int32)]


class DeltaTokens(C.Structure):
    _fields_ = [("q", vp), ("k", vp), ("v", vp), ("g", vp), ("beta", vp), ("q_stride", C.c_int64),
                ("k_stride", C.c_int64), ("v_stride", C.c_int64), ("g_stride", C.c_int64),
                ("beta_stride", C.c_int64), ("tokens", C.c_int64), ("scale", C.c_float)]


class DeltaGrads(C.Structure):
    _fields_ = [("dq", vp), ("dk", vp), ("dv", vp), ("dg", vp), ("dbeta", vp), ("q_stride", C.c_int64),
                ("k_stride", C.c_int64), ("v_stride", C.c_int64), ("g_stride", C.c_int64),
                ("beta_stride", C.c_int64)]


# struct formats of ofrl_delta_tokens and ofrl_delta_grads: packing one is several times cheaper than filling a
# ctypes Structure, and a call on one token costs little else on the host
DELTA_TOKENS_FMT = "5Q6qf4x"
DELTA_GRADS_FMT = "5Q5q"

ACT_NONE, ACT_SILU = 0, 1


class ConvShape(C.Structure):
    _fields_ = [("channels", C.c_int32), ("width", C.c_int32), ("activation", C.c_int32), ("dtype", C.c_int32)]


class ConvTokens(C.Structure):
    _fields_ = [("x", vp), ("weight", vp), ("bias", vp), ("x_stride", C.c_int64), ("tokens", C.c_int64)]


class ConvGrads(C.Structure):
    _fields_ = [("dx", vp), ("dweight", vp), ("dbias", vp), ("x_stride", C.c_int64)]


class ScanShape(C.Structure):
    _fields_ = [("channels", C.c_int32), ("state_dim", C.c_int32), ("groups", C.c_int32), ("dtype", C.c_int32),
                ("softplus", C.c_int32)]


class ScanTokens(C.Structure):
    _fields_ = [("x", vp), ("dt", vp), ("b", vp), ("c", vp), ("z", vp), ("a", vp), ("d", vp), ("dt_bias", vp),
                ("x_stride", C.c_int64), ("dt_stride", C.c_int64), ("b_stride", C.c_int64), ("c_stride", C.c_int64),
                ("z_stride", C.c_int64), ("tokens", C.c_int64)]


class ScanGrads(C.Structure):
    _fields_ = [("dx", vp), ("ddt", vp), ("db", vp), ("dc", vp), ("dz", vp), ("da", vp), ("dd", vp), ("ddt_bias", vp),
                ("x_stride", C.c_int64), ("dt_stride", C.c_int64), ("b_stride", C.c_int64), ("c_stride", C.c_int64),
                ("z_stride", C.c_int64)]


class NormShape(C.Structure):
    _fields_ = [("channels", C.c_int32), ("groups", C.c_int32), ("dtype", C.c_int32), ("residual_dtype", C.c_int32)]


class GatedRows(C.Structure):
    _fields_ = [("x", vp), ("z", vp), ("weight", vp), ("x_stride", C.c_int64), ("z_stride", C.c_int64),
                ("rows", C.c_int64), ("eps", C.c_float), ("gate_first", C.c_int32)]


class ResidualRows(C.Structure):
    _fields_ = [("x", vp), ("residual", vp), ("scale", vp), ("weight", vp), ("x_stride", C.c_int64),
                ("residual_stride", C.c_int64), ("rows", C.c_int64), ("eps", C.c_float)]


CONV_TOKENS_FMT = "3Q2q"
CONV_GRADS_FMT = "3Qq"
SCAN_TOKENS_FMT = "8Q6q"
SCAN_GRADS_FMT = "8Q5q"
GATED_ROWS_FMT = "3Q3qfi"
RESIDUAL_ROWS_FMT = "4Q3qf4x"

# name -> (restype, argtypes)
SIGNATURES = {
    "ofrl_create": (C.c_int32, [C.POINTER(VShape), C.c_int32, C.c_int32, C.POINTER(vp)]),
    "ofrl_destroy": (C.c_int32, [vp]),
    "ofrl_poll_status": (C.c_int32, [vp, vp, C.POINTER(C.c_int32)]),
    "ofrl_status_string": (C.c_char_p, [C.c_int32]),
    "ofrl_workspace_bytes": (C.c_int64, [C.POINTER(VShape), C.c_int32, C.c_int32]),
    "ofrl_her_relabel": (C.c_int32, [vp, C.POINTER(Replay), C.POINTER(HerCfg), C.c_uint64, C.POINTER(Batch), vp]),
    "ofrl_her_relabel_sources": (C.c_int32, [vp, C.POINTER(Replay), C.POINTER(HerCfg), C.c_uint64, vp, vp,
                                             C.POINTER(Batch), vp, vp]),
    "ofrl_episode_ends_append": (C.c_int32, [vp, vp, C.c_int64, C.c_int32, vp, vp, C.c_int32, vp]),
    "ofrl_iql_value_fwd_bwd": (C.c_int32, [vp, vp, vp, C.c_int32, C.c_int32, vp, C.c_float, vp, vp, vp, vp]),
    "ofrl_forward_values": (C.c_int32, [vp, vp, vp, C.c_int32, C.c_int32, vp, vp]),
    "ofrl_iql_target": (C.c_int32, [vp, vp, vp, C.c_int32, vp, vp, C.c_int32, C.c_float, vp, vp, vp]),
    "ofrl_expectile_loss": (C.c_int32, [vp, vp, vp, C.c_int32, C.c_float, vp, vp, vp]),
    "ofrl_adv_weighted_policy": (C.c_int32, [vp, vp, vp, C.c_int32, C.c_int32, C.c_float, vp, vp, vp]),
    "ofrl_budgeted_clip_saxpy": (C.c_int32, [vp, C.POINTER(vp), C.POINTER(C.c_float), C.POINTER(C.c_float),
                                             C.c_int32, C.c_int64, C.c_float, vp, vp, vp]),
    "ofrl_target_ema": (C.c_int32, [vp, vp, C.c_int64, C.c_float, vp]),
    "ofrl_adam_step": (C.c_int32, [vp, vp, vp, vp, vp, C.c_int64, C.c_int32, C.POINTER(Opt), vp, vp]),
    "ofrl_train_step": (C.c_int32, [vp, C.POINTER(Replay), C.POINTER(HerCfg), C.c_uint64, C.POINTER(Batch), vp,
                                    C.POINTER(VNet), C.c_int32, C.POINTER(Opt), C.POINTER(vp), C.c_int32,
                                    vp, vp, vp, vp, vp, vp, vp]),
    "ofrl_train_step_kernels": (C.c_int32, [vp, C.POINTER(Batch), C.c_int32, C.c_int32]),
    "ofrl_select_vnet_path": (C.c_int32, [vp, C.c_int32]),
    "ofrl_vnet_path": (C.c_int32, [vp, C.c_int32]),
    "ofrl_step_graph_create": (C.c_int32, [vp, C.POINTER(Replay), C.POINTER(HerCfg), C.POINTER(Batch), vp, vp,
                                           C.c_int32, C.POINTER(Opt), C.POINTER(vp), C.c_int32, vp, vp, vp, vp, vp,
                                           vp, C.POINTER(vp)]),
    "ofrl_step_graph_launch": (C.c_int32, [vp, C.c_uint64, vp, C.POINTER(vp), vp]),
    "ofrl_step_graph_destroy": (C.c_int32, [vp]),
    "ofrl_step_graph_create_io": (C.c_int32, [vp, C.POINTER(Replay), C.POINTER(HerCfg), C.POINTER(Batch), vp, vp,
                                              C.c_int32, C.POINTER(Opt), C.POINTER(vp), C.c_int32, vp, vp, vp, vp,
                                              vp, vp, vp, vp, vp, C.POINTER(vp)]),
    "ofrl_step_graph_launch_io": (C.c_int32, [vp, C.c_uint64, vp, C.POINTER(vp), vp, vp, vp]),
    "ofrl_noalloc_max_batch": (C.c_int64, [C.POINTER(VShape)]),
    "ofrl_iql_value_fwd_bwd_noalloc": (C.c_int32, [C.POINTER(VShape), vp, vp, C.c_int32, C.c_int32, vp, C.c_float,
                                                   vp, vp, vp, vp]),
    "ofrl_selftest_umma": (C.c_int32, [vp, vp, vp, C.c_int32, C.c_int32, C.c_int32, C.c_int32, C.c_int32,
                                       C.c_int32, vp, vp]),
    "ofrl_selftest_barrier": (C.c_int32, [vp, C.c_uint64, C.c_int32]),
    "ofrl_selftest_scan_cut": (C.c_int32, [vp, C.c_int64, C.c_int32, C.c_int64, C.c_int32, C.c_int32, vp]),
    "ofrl_delta_create": (C.c_int32, [C.POINTER(DeltaShape), C.c_int64, C.c_int32, C.c_int32, C.POINTER(vp)]),
    "ofrl_delta_destroy": (C.c_int32, [vp]),
    "ofrl_delta_poll_status": (C.c_int32, [vp, vp, C.POINTER(C.c_int32)]),
    "ofrl_delta_workspace_bytes": (C.c_int64, [C.POINTER(DeltaShape), C.c_int64, C.c_int32, C.c_int32]),
    "ofrl_delta_saved_bytes": (C.c_int64, [C.POINTER(DeltaShape), C.c_int64, C.c_int32]),
    # token and gradient structs are passed as packed bytes (see DELTA_TOKENS_FMT)
    "ofrl_delta_forward": (C.c_int32, [vp, C.c_char_p, vp, C.c_int32, vp, vp, vp, vp, vp]),
    "ofrl_delta_backward": (C.c_int32, [vp, C.c_char_p, vp, C.c_int32, vp, vp, vp, C.c_char_p, vp, vp]),
    "ofrl_delta_step": (C.c_int32, [vp, C.c_char_p, vp, C.c_int32, vp, vp, vp, vp]),
    "ofrl_tensors_create": (C.c_int32, [C.POINTER(vp), C.POINTER(C.c_int64), C.POINTER(C.c_int32), C.c_int32,
                                        C.POINTER(vp)]),
    "ofrl_tensors_destroy": (C.c_int32, [vp]),
    "ofrl_global_norm": (C.c_int32, [vp, vp, vp]),
    "ofrl_global_norm_clip": (C.c_int32, [vp, C.c_float, vp, vp, vp]),
    # token, row and gradient structs as packed bytes, as above
    "ofrl_conv_create": (C.c_int32, [C.POINTER(ConvShape), C.c_int64, C.c_int32, C.c_int32, C.POINTER(vp)]),
    "ofrl_conv_destroy": (C.c_int32, [vp]),
    "ofrl_conv_poll_status": (C.c_int32, [vp, vp, C.POINTER(C.c_int32)]),
    "ofrl_conv_workspace_bytes": (C.c_int64, [C.POINTER(ConvShape), C.c_int64, C.c_int32, C.c_int32]),
    "ofrl_conv_forward": (C.c_int32, [vp, C.c_char_p, vp, C.c_int32, vp, vp, C.c_int64, vp, vp]),
    "ofrl_conv_backward": (C.c_int32, [vp, C.c_char_p, vp, C.c_int32, vp, vp, C.c_int64, vp, C.c_char_p, vp, vp]),
    "ofrl_conv_step": (C.c_int32, [vp, C.c_char_p, vp, C.c_int32, vp, vp, vp, C.c_int64, vp]),
    "ofrl_scan_create": (C.c_int32, [C.POINTER(ScanShape), C.c_int64, C.c_int32, C.c_int32, C.POINTER(vp)]),
    "ofrl_scan_destroy": (C.c_int32, [vp]),
    "ofrl_scan_poll_status": (C.c_int32, [vp, vp, C.POINTER(C.c_int32)]),
    "ofrl_scan_workspace_bytes": (C.c_int64, [C.POINTER(ScanShape), C.c_int64, C.c_int32, C.c_int32]),
    "ofrl_scan_saved_bytes": (C.c_int64, [C.POINTER(ScanShape), C.c_int64]),
    "ofrl_scan_forward": (C.c_int32, [vp, C.c_char_p, vp, C.c_int32, vp, vp, C.c_int64, vp, vp, vp]),
    "ofrl_scan_backward": (C.c_int32, [vp, C.c_char_p, vp, C.c_int32, vp, vp, vp, C.c_int64, vp, C.c_char_p, vp, vp]),
    "ofrl_scan_step": (C.c_int32, [vp, C.c_char_p, vp, C.c_int32, vp, vp, vp, C.c_int64, vp]),
    "ofrl_norm_create": (C.c_int32, [C.POINTER(NormShape), C.c_int32, C.POINTER(vp)]),
    "ofrl_norm_destroy": (C.c_int32, [vp]),
    "ofrl_norm_workspace_bytes": (C.c_int64, [C.POINTER(NormShape), C.c_int32]),
    "ofrl_gated_norm": (C.c_int32, [vp, C.c_char_p, vp, C.c_int64, vp]),
    "ofrl_gated_norm_backward": (C.c_int32, [vp, C.c_char_p, vp, C.c_int64, vp, C.c_int64, vp, C.c_int64, vp, vp]),
    "ofrl_residual_norm": (C.c_int32, [vp, C.c_char_p, vp, C.c_int64, vp, C.c_int64, vp]),
    "ofrl_residual_norm_backward": (C.c_int32, [vp, C.c_char_p, vp, C.c_int64, vp, C.c_int64, vp, C.c_int64, vp,
                                                C.c_int64, vp, vp, vp]),
    "ofrl_profile_begin": (C.c_int32, [vp, C.c_int32]),
    "ofrl_profile_end": (C.c_int32, [vp, C.POINTER(C.c_float), C.POINTER(C.c_int32)]),
}
PHASES = ("relabel", "vnet", "reduce", "adam")

_LIB = None


class OfrlError(RuntimeError):
    def __init__(self, fn, code, msg):
        super().__init__(f"{fn} failed: {msg} ({code})")
        self.code = code


def load(path: str = LIB_PATH):
    """Load libofrl.so (built by offline_rl_step_gb300.build) and declare its symbols."""
    global _LIB
    if _LIB is not None:
        return _LIB
    if not os.path.exists(path):
        raise RuntimeError(
            f"the ofrl CUDA library is not built ({path} is missing); run "
            "`python -m offline_rl_step_gb300.build` or __graft_entry__.build() first")
    lib = C.CDLL(path)
    for name, (res, args) in SIGNATURES.items():
        fn = getattr(lib, name)
        fn.restype = res
        fn.argtypes = args
    _LIB = lib
    return lib


def check(fn: str, code: int):
    if code != OK:
        msg = load().ofrl_status_string(code).decode()
        raise OfrlError(fn, code, msg)
