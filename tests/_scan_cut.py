"""How the selective scan cuts a call, and calls whose segments are whole episodes."""
import collections
import ctypes as C

Cut = collections.namedtuple("Cut", "lanes each blocks seg segments used held")

# shape, episodes, their length, gradients, channels of a thread: the wide form, the narrow one before and after the
# wide one's even shares were looked at, and shapes whose only form is the narrow one
WHOLE = {
    "wide": ((200, 12, 1), 80, 80, False, 4),
    "wide, two channels": ((72, 8, 1), 160, 80, False, 2),
    "wide, 16 lanes": ((144, 64, 1), 32, 80, False, 4),
    "narrow, first": ((200, 12, 1), 24, 80, False, 1),
    "narrow, first, 8 lanes": ((128, 28, 1), 20, 80, False, 1),
    "narrow, last": ((72, 8, 1), 80, 112, False, 1),
    "narrow, last, 8 lanes": ((128, 28, 1), 20, 112, False, 1),
    "narrow, groups": ((48, 4, 3), 64, 80, False, 1),
    "production": ((128, 16, 1), 64, 256, False, 1),
    "gradients, wide": ((72, 12, 1), 160, 80, True, 4),
    "gradients, narrow": ((72, 12, 1), 80, 80, True, 2),
    "gradients, narrow, one channel": ((72, 8, 1), 80, 80, True, 1),
    "gradients, narrow, 16 lanes": ((40, 64, 1), 64, 80, True, 2),
    "gradients, groups": ((48, 4, 3), 64, 80, True, 1),
}


def cut_of(shape, tokens, episodes, sms, backward, max_tokens=None):
    """shape: channels, states, groups.  each: channels of a thread; used, held: bytes of workspace."""
    from offline_rl_step_gb300 import _abi
    out = (C.c_int64 * 7)()
    s = _abi.ScanShape(*shape, 1, 1)
    code = _abi.load().ofrl_selftest_scan_cut(C.byref(s), tokens, episodes, tokens if max_tokens is None else max_tokens,
                                              sms, int(backward), out)
    assert code == _abi.OK
    return Cut(*out)
