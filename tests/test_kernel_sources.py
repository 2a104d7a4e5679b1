"""Checks of the CUDA sources that no compiler flag of the build makes (CPU)."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "paged_kv_gqa_nx_gb300", "csrc")
FILES = sorted(f for f in os.listdir(CSRC) if f.endswith((".cu", ".cpp", ".h")))


def text(name):
    with open(os.path.join(CSRC, name)) as f:
        return re.sub(r"//[^\n]*|/\*.*?\*/", "", f.read(), flags=re.S)


def seen_by(name, done=None):
    """The file and the headers beside it that it includes."""
    done = set() if done is None else done
    if name not in done:
        done.add(name)
        for inc in re.findall(r'#include "([^"/]+)"', open(os.path.join(CSRC, name)).read()):
            seen_by(inc, done)
    return done


def constants(name):
    """Names of the constants at namespace scope (their declarations start a line)."""
    out = set()
    for decl in re.findall(r"^(?:static |inline )*constexpr [\w:]+ ([^;{(]*=[^;]*);", text(name), flags=re.M):
        out.update(re.findall(r"(?:^|,)\s*(k[A-Z]\w*)\s*=", decl))
    return out


def template_parameters(name):
    out = set()
    for params in re.findall(r"\btemplate\s*<([^<>]*(?:<[^<>]*>[^<>]*)*)>", text(name)):
        out.update(p.split("=")[0].split()[-1] for p in params.split(",") if p.split("=")[0].split())
    return out


def test_the_scan_finds_what_it_looks_for():
    assert "kFull" in constants("pkv_rows.h") and {"kW", "kT"} <= constants("pkv_q8.cu")
    assert {"kVec", "S", "E", "B"} <= template_parameters("pkv_pages.cu")


@pytest.mark.parametrize("name", FILES)
def test_no_template_parameter_hides_a_constant(name):
    """A parameter of a constant's name takes its place without a word: a lane mask became a truth value once."""
    known = set().union(*(constants(f) for f in seen_by(name)))
    assert not known & template_parameters(name)
