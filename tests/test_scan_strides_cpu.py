"""The selective scan's forward reaches the rows of a block of tokens from its first one by 32
bits.  Which kernel a call takes, and so how many rows its blocks have, is seen without a GPU:
the calls run in a process of their own in which a library made here stands in for the HIP
runtime's beginning of a launch and writes down the sizes of the workgroups."""
import json
import os
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
LIB = os.path.join(ROOT, "cfc_recurrent_cell_amd", "libcfc_amd.so")
pytestmark = pytest.mark.skipif(not os.path.exists(LIB), reason="libcfc_amd.so not built (run __graft_entry__.build())")

RECORDER = """
struct size { unsigned x, y, z; };
unsigned launched_threads, launches;
int __hipPushCallConfiguration(struct size grid, struct size block, unsigned long shared, void *stream) {
    launched_threads = block.x;
    ++launches;
    return 1; /* nothing is launched */
}
int hipGetLastError(void) { return 0; }
"""
CHANNELS, TOKENS = 64, 300
STRIDES = ("x_stride", "dt_stride", "z_stride", "b_stride_t", "c_stride_t")
STATES = (1, 4, 5, 8, 9, 16, 17, 32, 33, 64)


def tokens_of_a_wave(state):
    return 8 if state <= 8 else 4


def calls(recorder):
    """For each type, state and stride: the largest one that is accepted, and the threads of the
    forward's workgroups there, at half and at a quarter of it."""
    import ctypes
    seen = ctypes.CDLL(recorder, mode=ctypes.RTLD_GLOBAL)
    sys.path.insert(0, ROOT)
    from cfc_recurrent_cell_amd import _lib
    lib = _lib.load_library()
    threads = ctypes.c_uint.in_dll(seen, "launched_threads")
    count = ctypes.c_uint.in_dll(seen, "launches")
    out = []
    for kind, size in ((_lib.CFC_TYPE_F32, 4), (_lib.CFC_TYPE_BF16, 2), (_lib.CFC_TYPE_F16, 2)):
        for state in STATES:
            dense = dict(x_stride=CHANNELS, dt_stride=CHANNELS, z_stride=CHANNELS, grad_y_stride=CHANNELS, b_stride_t=state,
                         b_stride_g=state, c_stride_t=state, c_stride_g=state)

            def shape(**over):
                return _lib.SelectiveScanShape(kind, 1, TOKENS, TOKENS, None, CHANNELS, 1, state, 1, 0, *{**dense, **over}.values())

            def forward(**over):
                before, far = count.value, 1 << 44
                code = lib.selective_scan_forward(ctypes.byref(shape(**over)), *[far * (i + 1) for i in range(11)], None)
                assert code == 0 and count.value == before + 1, (code, over)
                return threads.value

            for name in STRIDES:
                low, high = 1, 1 << 40
                while high - low > 1:
                    middle = (low + high) // 2
                    if lib.selective_scan_backward_workspace(ctypes.byref(shape(**{name: middle}))) >= 0:
                        low = middle
                    else:
                        high = middle
                out.append(dict(size=size, state=state, stride=name, most=low, dense=forward(),
                                threads=[(s, forward(**{name: s})) for s in (low, low // 2 + 1, low // 2 - CHANNELS - state, low // 4)]))
    print(json.dumps(out))


@pytest.fixture(scope="module")
def seen(tmp_path_factory):
    at = tmp_path_factory.mktemp("recorder")
    source, recorder = str(at / "recorder.c"), str(at / "recorder.so")
    with open(source, "w") as f:
        f.write(RECORDER)
    subprocess.run(["gcc", "-shared", "-fPIC", "-o", recorder, source], check=True)
    done = subprocess.run([sys.executable, os.path.abspath(__file__), recorder], check=True, stdout=subprocess.PIPE, timeout=300)
    return json.loads(done.stdout.decode().splitlines()[-1])


def test_rows_of_a_block_are_within_31_bits(seen):
    assert len(seen) == 3 * len(STATES) * len(STRIDES)
    for case in seen:
        width = max(CHANNELS, case["state"]) * case["size"]
        for stride, threads in case["threads"]:
            rows = threads // 64 * tokens_of_a_wave(case["state"])
            assert rows * stride * case["size"] + width < 1 << 31, (case, stride, threads, rows)


def test_64_rows_are_accepted_and_few_workgroups_have_16_waves_where_theirs_reach(seen):
    for case in seen:
        assert 64 * (case["most"] + CHANNELS + case["state"]) * case["size"] >= (1 << 31) - 64 * case["size"], case
        assert case["dense"] == case["threads"][-1][1], case  # a quarter of the longest stride is like a dense one


if __name__ == "__main__":
    calls(sys.argv[1])
