"""The roles of the attention kernels on the host: their source, cut out of the kernels' files and compiled with a fiber
per thread (attn_roles_host.h).  Whichever wait of whichever warp runs out, all threads come to their end; between a
thread's write of a shared entry and another's access to it there is a barrier that both pass; and a role that ends
has waited for the copies and MMAs under way, however short the limit on waits is."""
import os
import re
import shutil
import subprocess

import pytest

from lightning_attention_gb300 import _build

HERE = os.path.dirname(os.path.abspath(__file__))
pytestmark = pytest.mark.skipif(shutil.which("g++") is None, reason="no host compiler")


def source(name):
    with open(os.path.join(_build.CSRC, name)) as f:
        return re.sub(r"//[^\n]*", "", f.read())


def cut(text, pattern):
    """The definition that begins with `pattern` at the start of a line, with the template line before it."""
    m = re.search(r"^(?:template <[^\n]*>\n)?" + pattern, text, re.M)
    assert m, pattern
    depth, i = 0, text.index("{", m.end())
    while True:
        depth += {"{": 1, "}": -1}.get(text[i], 0)
        i += 1
        if depth == 0:
            break
    return text[m.start():i] + (";" if pattern.startswith("struct") else "") + "\n"


def constants(text, *names):
    return "\n".join(re.search(rf"^constexpr [^;]*\b{n} = [^;]*;", text, re.M).group(0) for n in names) + "\n"


def function(name):
    return rf"[^\n(]*\b{name}\("


def build(tmp_path, parts):
    src, exe = tmp_path / "roles.cc", tmp_path / "roles"
    src.write_text('#include "attn_roles_host.h"\n' + "\n".join(parts))
    # what nobody has set holds a pattern
    subprocess.run(["g++", "-std=c++17", "-O1", "-w", "-ftrivial-auto-var-init=pattern", "-I", HERE, str(src),
                    "-o", str(exe)], check=True)
    return str(exe)


def runs(exe, *args):
    r = subprocess.run([exe, *map(str, args)], capture_output=True, text=True, timeout=120)
    assert r.returncode == 0, r.stdout + r.stderr


def common():
    h = source("la_attn.h")
    internal, t = source("la_internal.h"), source("la_attn.cuh")
    return [constants(internal, "kHeadDim"), "typedef int cudaStream_t;\n", cut(internal, r"enum : unsigned int"), ";",
            constants(h, "kVerifyRows", "kAttnCtas", "kMaxDrafts", "kKeyTile"), cut(h, "struct CacheParams"),
            cut(h, "struct AttnParams"), constants(t, "kTileBytes", "kHalfBytes"),
            "".join(re.findall(r"^constexpr uint64_t kDrainLimitNs[^;]*;", t, re.M)), cut(t, "struct Waiter"),
            cut(t, function("page_shift")), cut(t, "struct Pages"), cut(t, function("load_tile")),
            cut(t, function("group_size")), cut(t, function("scan_lanes")), cut(t, "struct Place"),
            cut(t, "struct Runs"), cut(t, "struct Tail")]


PART = r"""
enum { SOFTMAX, LOADS, VALUES, MMAS };
static int part;
static uint8_t smem[1 << 18];
"""
MAIN = r"""
static uint8_t *page(size_t n) { return static_cast<uint8_t *>(calloc(n, 1)); }
int main(int argc, char **argv) {
    part = atoi(argv[1]);
    rising = atoi(argv[2]);
    const int lens[] = {300};
    const int32_t parents[] = {-1, 0, 0, -1};
    AttnParams p = {};
    p.cache.kv_lens = lens;
    p.cache.page_size = 16;
    p.cache.max_pages = 100;
    p.out = reinterpret_cast<__nv_bfloat16 *>(page(1 << 20));
    p.ws = page(4 << 20);
    unsigned err = 0;
    p.err = &err;
    p.scale_log2 = 1.f;
    p.B = 1;
    p.H = 4;
    p.Hkv = 2;
    p.group = 2;
    p.N = 4;
    p.T = 300;
    p.split = 1;
    static int32_t table[100];
    p.cache.page_table = table;
    p.cache.num_pages = 1;
    const bool tree = atoi(argv[3]);
    if (tree) p.parents = parents;
    Bars_ *bars = reinterpret_cast<Bars_ *>(page(sizeof(Bars_)));
    // items by the tiles that each has, at most three
    static const int items[][3] = {{1}, {3}, {1, 2, 1}, {2, 2}};
    for (const auto &tiles : items) {
        char name[64];
        snprintf(name, sizeof name, "items of %d, %d, %d tiles", tiles[0], tiles[1], tiles[2]);
        scenario = name;
        const std::vector<int> all = WARPS, some = RUN_OUT, one = {0};
        every_wait(part == SOFTMAX ? all : one, part == SOFTMAX ? some : one, [&]() {
            if (self == &fibers[0]) {
                memset(bars, 0, sizeof *bars);
                for (int i = 0; i < 3; ++i) set_item(bars, i, tiles[i], parents);
            }
            role(p, bars);
        });
    }
    return 0;
}
"""


@pytest.fixture(scope="module")
def prompts(tmp_path_factory):
    t = source("la_attn_extend.cu")
    bars = cut(t, "struct Bars").replace("float swap", "Cell swap")
    assert "Cell swap" in bars
    parts = common() + [constants(t, "kRowTile", "kItemRows", "kSlots", "kMmaWarp", "kItems", "kPieceFloats"),
                        cut(t, "struct Rec"), constants(t, "kNoParent"), bars, constants(t, "kTmS", "kUnseen")]
    parts += [cut(t, function(n)) for n in ("columns_seen", "drafts_seen", "mask_scores", "largest", "exponents", "weigh")]
    parts += [r"""
static int named_place(int id) { return (threadIdx.x >> 7 & 1) * 32 + lane_of(); }
static int named_count(int id) { return 64; }
static bool pair_any(int pair, bool x) { return named_any(pair + 1, x); }
""", cut(t, function("quad_transpose")), cut(t, function("softmax_role")), constants(t, "kOffQ", "kOffKV"),
              cut(t, "struct Request"), cut(t, function("request_of")), constants(t, "kItemKeys")]
    parts += [cut(t, function(n)) for n in ("work_of", "cut", "tokens_of", "items_of", "request_work")]
    parts += [cut(t, "struct Item"), cut(t, "struct Walk"), cut(t, "struct Ring")]
    parts += [cut(t, function(n)) for n in ("drain_ring", "parents_of", "load_role", "value_role", "mma_role")] + [PART, r"""
using Bars_ = Bars;
#define WARPS {1, 5}
#define RUN_OUT WARPS
static void set_item(Bars *bars, int i, int tiles, const int32_t *parents) {
    Rec &r = bars->items[i];
    memset(bars->parent[i], kNoParent, kMaxDrafts);
    for (int t = 0; t < 4; ++t)
        if (parents[t] >= 0) bars->parent[i][t] = (uint8_t)parents[t];
    r.n = 4;
    r.kv_len = 300;
    r.j1 = tiles;
    r.whole = i != 1;
    r.sound = 1;
}
static void role(const AttnParams &p0, Bars *bars) {
    AttnParams p = p0;
    static const int32_t cu[] = {0, 4};
    const Waiter wait{1000, p.err};
    if (!p.parents) p.cu_seqlens = cu;
    if (part == LOADS) {
        if (self == &fibers[0]) bars->work[0] = request_work(p, 0, tokens_of(p), false);
        if (p.parents)
            load_role<true>(p, nullptr, nullptr, bars, smem, lane_of(), wait);
        else
            load_role<false>(p, nullptr, nullptr, bars, smem, lane_of(), wait);
        drain_ring(bars, wait);
    } else if (part == VALUES) {
        value_role(p, nullptr, bars, smem, lane_of(), wait);
        drain_ring(bars, wait);
    } else if (part == MMAS) {
        mma_role(p, bars, smem, 0, lane_of(), wait);
    } else
    if (p.parents)
        softmax_role<true>(p, bars, 0, threadIdx.x >> 5, lane_of(), wait);
    else
        softmax_role<false>(p, bars, 0, threadIdx.x >> 5, lane_of(), wait);
}
""", MAIN]
    return build(tmp_path_factory.mktemp("prompts"), parts)


@pytest.fixture(scope="module", params=[16, 64])
def few_rows(request, tmp_path_factory):
    t = source("la_attn_verify.cu")
    bars = cut(t, "struct Bars")
    for entry in ("float neg_m", "float factor", "float top"):
        assert entry in bars
        bars = bars.replace(entry, entry.replace("float", "Cell"))
    role = cut(t, function("softmax_role"))
    vector = "*reinterpret_cast<const float4 *>(&bars->neg_m[r0 + r])"
    assert role.count(vector) == 1
    parts = common() + [constants(t, "kMmaWarp", "kMaxRuns", "kUnseen"), cut(t, "struct Shape"), cut(t, "struct Rec"),
                        constants(t, "kItems"), bars, cut(t, function("tiles_of")), r"""
static int named_place(int id) { return threadIdx.x; }
static int named_count(int id) { return 256; }
static bool softmax_any(bool x) { return named_any(1, x); }
static void softmax_sync() { named_any(1, false); }
""", cut(t, function("build_tree")), role.replace(vector, "load4(&bars->neg_m[r0 + r])")]
    parts += [cut(t, function(n)) for n in ("work_of", "cut", "request_work")] + [cut(t, "struct Walk"), cut(t, "struct Ring")]
    parts += [cut(t, function(n)) for n in ("drain_ring", "load_role", "value_role", "mma_role")] + [PART, r"""
constexpr int RP = %d;
using Bars_ = Bars<RP>;
#define WARPS {0, 1, 2, 3, 4, 5, 6, 7}
#define RUN_OUT {0, 6}
static void set_item(Bars_ *bars, int i, int tiles, const int32_t *) {
    Rec &r = bars->items[i];
    r.kv_len = 300;
    r.j1 = tiles;
    r.whole = i != 1;
}
static void role(const AttnParams &p, Bars_ *bars) {
    const Waiter wait{1000, p.err};
    if (part == LOADS) {
        if (self == &fibers[0]) bars->work[0] = request_work(p, 0, Shape<RP, 1>::kExtra);
        load_role<RP, 1>(p, nullptr, nullptr, bars, smem, lane_of(), wait);
        const Tail &t = *static_cast<Tail *>(p.ws);
        if (t.tiles == 0 && (t.at || t.size || t.b || t.kvh)) broken("a record of no item holds something", t.b, t.kvh);
        drain_ring<RP, 1>(bars, wait);
        return;
    }
    if (part == VALUES) {
        value_role<RP, 1>(p, nullptr, bars, smem, lane_of(), wait);
        drain_ring<RP, 1>(bars, wait);
        return;
    }
    if (part == MMAS) return mma_role<RP, 1>(p, bars, smem, 0, lane_of(), wait);
    for (int r = lane_of(); r < RP; r += 32) bars->tok_of[r] = (uint8_t)(r / p.group);
    softmax_role<RP, 1>(p, bars, smem, 0, threadIdx.x >> 5, lane_of(), wait);
}
""" % request.param, MAIN]
    return build(tmp_path_factory.mktemp("few"), parts)


SOFTMAX, LOADS, VALUES, MMAS = range(4)


@pytest.mark.parametrize("part", [LOADS, VALUES, MMAS])
@pytest.mark.parametrize("tree", [0, 1])
def test_what_is_under_way_is_waited_for(prompts, few_rows, part, tree):
    for exe in (prompts, few_rows):
        runs(exe, part, 0, tree)


@pytest.mark.parametrize("rising", [0, 1])
@pytest.mark.parametrize("tree", [0, 1])
def test_prompt_role(prompts, rising, tree):
    runs(prompts, SOFTMAX, rising, tree)


@pytest.mark.parametrize("rising", [0, 1])
@pytest.mark.parametrize("tree", [0, 1])
def test_role_of_few_rows(few_rows, rising, tree):
    runs(few_rows, SOFTMAX, rising, tree)
