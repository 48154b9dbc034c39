"""Kernels that are launched as programmatic dependents (they call wait_previous()) may be resident while the kernel
before them still writes what they read. The non-coherent path (ld.global.nc) is only for memory that nobody writes
while the kernel lives, so such kernels use no ld_stream, no __ldg and no `const T *__restrict__` (from which the compiler
makes non-coherent loads by itself). Read from the source, no GPU needed."""
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "mixture_experts_layer_histogram_gb300",
                    "csrc")


def source(name):
    with open(os.path.join(CSRC, name)) as f:
        return re.sub(r"//[^\n]*", "", f.read())


def braced(text, at):
    """From `at` to the end of the first brace-delimited block that begins after it."""
    i = text.index("{", at)
    depth = 0
    for j in range(i, len(text)):
        depth += {"{": 1, "}": -1}.get(text[j], 0)
        if depth == 0:
            return text[at:j + 1]
    raise AssertionError("unbalanced braces")


def kernels():
    """(file, name, text) of every kernel that waits for the one before it."""
    for name in sorted(os.listdir(CSRC)):
        text = source(name)
        for m in re.finditer(r"__global__", text):
            body = braced(text, m.start())
            if "wait_previous()" in body:
                yield name, re.search(r"(\w+_kernel)\s*\(", body).group(1), body


def functions(name):
    """Device functions of a file and of the headers, by name."""
    found = {}
    for file in [name] + [n for n in os.listdir(CSRC) if n.endswith(".cuh")]:
        text = source(file)
        for m in re.finditer(r"__device__ __forceinline__ [\w<> ]*?[ *&]*(\w+)\s*\(", text):
            found.setdefault(m.group(1), braced(text, m.start()))
    return found


def test_dependent_kernels_read_coherently():
    seen = set()
    for file, kernel, body in kernels():
        seen.add(kernel)
        known = functions(file)
        todo, done = [kernel], set()
        texts = {kernel: body}
        while todo:
            text = texts[todo.pop()]
            for f in set(re.findall(r"(\w+)\s*(?:<[^;()]*>)?\s*\(", text)) & set(known) - done:
                done.add(f)
                texts[f] = known[f]
                todo.append(f)
        for f, text in texts.items():
            assert "ld.global.nc" not in text and "__ldg(" not in text, (file, kernel, f)
        for arg in re.findall(r"const\s+\w+\s*\*\s*__restrict__\s+\w+", body):
            raise AssertionError((file, kernel, arg))
    assert {"combine_kernel", "fp4_kernel", "fp4_few_kernel", "norm_bwd_sum_kernel"} <= seen
