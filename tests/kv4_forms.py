"""Which form of the attention a call takes, from the kernels' own header: the
waves of a workgroup share rows and split tokens ("few"), or own rows ("many")."""
import collections
import ctypes
import functools
import os
import subprocess
import tempfile

from ternary_packed_weight_amd import build

SOURCE = r'''
#include "tq2_kv4.h"
extern "C" {
void plan(int Hq, int Hk, int D, int P, int width, int B, int max_q, int window, int* o) {
  const tq2::Kv4AttnPlan p = tq2::plan_kv4_attn(Hq, Hk, D, P, width, B, max_q, window);
  o[0] = p.few, o[1] = p.mt, o[2] = p.list, o[3] = p.budget, o[4] = p.least, o[5] = p.rows, o[6] = p.tiles;
}
void part(int tiles, int parts, int part, int step, int* o) {
  const tq2::Kv4Part p = tq2::kv4_part(tiles, parts, part, step);
  o[0] = p.first, o[1] = p.last;
}
}
'''
Plan = collections.namedtuple("Plan", "few mt list budget least rows tiles")


@functools.lru_cache(None)
def _lib():
    with tempfile.TemporaryDirectory() as d:
        src, so = os.path.join(d, "forms.cpp"), os.path.join(d, "forms.so")
        with open(src, "w") as f:
            f.write(SOURCE)
        subprocess.run(["g++", "-std=c++17", "-O1", "-shared", "-fPIC", "-Wall", "-Werror", "-I", build.CSRC, src, "-o", so],
                       check=True)
        return ctypes.CDLL(so)


def plan(Hq, Hk, D, P, width, B, max_q, window=0):
    o = (ctypes.c_int * 7)()
    _lib().plan(Hq, Hk, D, P, width, B, max_q, window, o)
    return Plan(bool(o[0]), o[1], bool(o[2]), *o[3:])


def part(tiles, parts, i, step):
    o = (ctypes.c_int * 2)()
    _lib().part(tiles, parts, i, step, o)
    return o[0], o[1]


def kept(few):
    """What a probability times its token's scale is rounded to: the remainder's 22 bits, or one rounding to binary16."""
    return 2.0 ** -22 if few else 2.0 ** -11
