"""CPU check of the kernels' shared-memory barriers, from the source: every
barrier that a kernel initialises has a place of its own within the area that
its layout reserves (behind it lie the tensor-memory base and the abort flag)."""
import glob
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "fixed_pattern_sparse_sa_b200", "csrc")
_STEP = re.compile(r"for \(int (\w+) = 0; \1 < ([^;]+); \+\+\1\)|mbar_init\(([^,]+),[^;]*\);")


def _source(path):
    return re.sub(r"//[^\n]*", "", open(path).read())


def _constants():
    env = {}
    for path in glob.glob(os.path.join(CSRC, "*.cuh")):
        for name, value in re.findall(r"constexpr int (\w+) = (\d+);", _source(path)):
            env[name] = int(value)
    return env


def _body(text, at):
    """The statement or block that starts at `at`; (its text, where it ends)."""
    while text[at].isspace():
        at += 1
    if text[at] != "{":
        end = text.index(";", at) + 1
        return text[at:end], end
    depth, end = 0, at
    while True:
        depth += (text[end] == "{") - (text[end] == "}")
        end += 1
        if depth == 0:
            return text[at + 1:end - 1], end


def _inits(text, env):
    out, at = [], 0
    while (m := _STEP.search(text, at)) is not None:
        if m.group(3):
            out.append(eval(m.group(3), {}, env))
            at = m.end()
            continue
        body, at = _body(text, m.end())
        if "mbar_init" in body:
            for i in range(eval(m.group(2), {}, env)):
                out += _inits(body, {**env, m.group(1): i})
    return out


def _kernels():
    env = _constants()
    for path in sorted(glob.glob(os.path.join(CSRC, "*.cuh"))):
        text = _source(path)
        areas = [eval(x, {}, env) for x in re.findall(r"constexpr int N_BAR = ([^;]+);", text)]
        starts = [m.start() for m in re.finditer(r"uint64_t \*bars = ", text)]
        if not areas:                                             # (a kernel that has no such layout)
            continue
        assert len(areas) == len(starts), path
        for i, (area, a) in enumerate(zip(areas, starts)):
            part = text[a:starts[i + 1] if i + 1 < len(starts) else len(text)]
            names = dict(env)
            for decl in re.findall(r"uint64_t (\*[^;]+);", part):
                for name, expr in re.findall(r"\*(\w+) = ([^,]+)", decl):
                    if name == "bars":
                        names[name] = 0
                    elif "(" not in expr:
                        names[name] = eval(expr, {}, names)
            yield pytest.param(area, _inits(part[:part.index("__syncthreads", part.index("mbar_init"))], names),
                               id=f"{os.path.basename(path)}-{i}")


@pytest.mark.parametrize("area,places", list(_kernels()))
def test_every_barrier_has_a_place_of_its_own(area, places):
    assert len(places) > 5
    assert len(set(places)) == len(places), sorted(places)
    assert min(places) == 0 and max(places) < area, f"barriers 0 .. {max(places)} in an area of {area}"
