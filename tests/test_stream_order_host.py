"""Kernels are launched so that they may become resident while the previous grid of the stream is
still at work. Read here from the sources: none allocates tensor memory before it has waited for that
grid, which may still have to allocate its own (the two would wait for each other without a bound),
and every kernel that is launched that way waits."""
import glob
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "gated_deltanet_linear_14_gb300", "csrc")
WAITS = ("pdl_begin();", "pdl_wait_only();", "griddepcontrol.wait;")


def without_comments(text):
    return re.sub(r"//[^\n]*|/\*.*?\*/", "", text, flags=re.S)


def kernels():
    """(name, body) of every kernel, the body from its first brace to the matching one."""
    for path in sorted(glob.glob(os.path.join(CSRC, "*.cu*"))):
        text = without_comments(open(path).read())
        for m in re.finditer(r"__global__\s+void\s+(?:__launch_bounds__\s*\([^)]*(?:\([^)]*\)[^)]*)*\)\s*)?"
                             r"(\w+)\s*\(", text):
            at = text.index("{", m.end())
            depth, end = 1, at + 1
            while depth:
                depth += {"{": 1, "}": -1}.get(text[end], 0)
                end += 1
            yield m.group(1), text[at:end]


def launched():
    names = set()
    for path in glob.glob(os.path.join(CSRC, "*.cu*")):
        names.update(re.findall(r"launch_pdl\(\s*(\w+)", without_comments(open(path).read())))
    return names


def first(body, words):
    return min((body.find(w) for w in words if w in body), default=None)


def test_tensor_memory_is_allocated_after_the_wait():
    found = 0
    for name, body in kernels():
        at = first(body, ("tmem_alloc(",))
        if at is None:
            continue
        found += 1
        wait = first(body, WAITS)
        assert wait is not None and wait < at, name
    assert found >= 4, found


def test_every_kernel_waits_for_the_previous_grid():
    bodies = dict(kernels())
    names = [n for n in launched() if n in bodies]
    assert len(names) >= 8, names
    for name in names:
        assert first(bodies[name], WAITS) is not None, name
