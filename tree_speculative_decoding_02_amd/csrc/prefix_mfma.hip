// prefix_mfma.hip - attention behind shared prefixes on the matrix cores, bf16 and fp32, head widths
// 64, 96 and 128.
//
// A group's sequences are neighbours, so their rows are neighbours too: with the G = H / H_kv query
// heads that share a key head they are one list of rows, all of which see all of the prefix, and the
// workgroups of windowed attention (window_rows.h, window_rows_f32.h) run over it as over the rows of
// one sequence without rows of its own keys. Beside them, in the same launch, run the workgroups of
// each sequence's own tokens. All leave unnormalised parts - sum, largest score, sum of weights - at
// [part][row][head], and a second kernel joins a row's parts.
//
// Measured, 32 query heads over 8 key heads of 128, bf16: 64 single tokens behind one prefix of 16384,
// with up to 512 cached of their own, 50 us (40 to 45, and 7 for the join; 2.6 TB/s of the bytes that each
// have to be read once, 350 TFLOP/s); 50 trees of up to 16 nodes, four prefixes of up to 8192 among
// them, 74 us (63 and 12), 79 to 82 where three batches take turns, and 63 then without tokens of their
// own; 4 tokens behind 1000 12 us, two launches and the chains within; two prompts of 8192 rows behind 8192
// 3.9 ms (850 TFLOP/s), 315 us of it the join, as their sums pass through memory like all others. Tokens
// and trees are bound by the prefix's workgroups, two a CU at most and of one form: each has 64 keys at a
// time through registers to LDS, then products and exponentials behind a barrier. Tried: the own tokens'
// workgroups first (59 against 45), touching the rows three tiles ahead (52).
#include "prefix_device.h"
#include "window_rows.h"
#include "window_rows_f32.h"
#include "launch.h"

namespace bole {

// A sequence's own tokens: everything windowed attention shows with a window of everything.
struct OwnKeys {
    const PrefixArgs &p;
    static constexpr bool kOwnRows = true, kSplit = true;
    __device__ __forceinline__ const WindowArgs &args() const { return p.w; }
    template <int MT>
    __device__ __forceinline__ bool find(int G, int slot, bool report, RowTile &t, uint64_t &mask, int &depth) const {
        return find_tile<MT>(p.w, G, slot, report, t, mask, depth);
    }
    __device__ __forceinline__ const int32_t *table(int b) const { return p.w.page_table + (size_t)b * p.w.s.max_pages; }
    __device__ __forceinline__ int pages_status(const RowTile &t, int, int) const { return bole::pages_status(p.w, t.b, t.len); }
};

struct GroupRanges {
    const PrefixArgs &p;
    __device__ __forceinline__ void load(int x, int &lo, int &hi, int &len, bool &bad) const {
        const int b0 = p.group_offsets[x], b1 = p.group_offsets[x + 1], B = p.w.s.B;
        bad |= b0 < 0 || b1 < b0 || b1 > B;
        lo = p.w.offsets[min(max(b0, 0), B)], hi = p.w.offsets[min(max(b1, 0), B)], len = p.prefix_len[x];
    }
};

// Which part of which of the prefixes' row tiles item x of a key head is. One prefix is in `most` parts.
// Several are cut, once their lengths are known, into parts of a like number of key tiles, so that there
// are `items` at most, and `most` of a prefix (64 tokens over five prefixes of up to 16384: 64 us, with
// as many parts of each, whatever its length, 86).
struct Deal {
    Slot tile;
    int slot, part, parts;
};

template <int MT>
__device__ __forceinline__ Deal deal(const PrefixArgs &p, int G, int x, int items, int most) {
    const GroupRanges ranges{p};
    const int lane = lane_id(), T = p.w.s.T;
    Deal r = {{false, true, 0, 0, 0, 0, 0}, 0, 0, 1};
    if (p.groups == 1) {  // as many parts as the call's sizes say
        bool bad = false;
        int lo, hi, len;
        ranges.load(0, lo, hi, len, bad);
        bad |= lo < 0 || hi < lo || hi > T;
        const int tiles = max(1, uniform((int)(((uint32_t)(hi - lo) * G + MT - 1) / MT)));
        r.part = uniform(x / tiles), r.slot = x - r.part * tiles, r.parts = most;
        r.tile = {!bad && r.part < most, !bad, 0, lo, hi - lo, 0, len};
        return r;
    }
    const int longest = (int)min(((int64_t)p.max_prefix_pages << p.w.s.page_shift), (int64_t)0x7fffffff);
    bool bad = false;
    int lo, hi, len, tiles, keys;  // of a group a lane: its rows and tokens, and both in tiles
    auto load = [&](int c) {
        ranges.load(min(c + lane, p.groups - 1), lo, hi, len, bad);
        bad |= lo < 0 || hi < lo || hi > T;
        const bool there = c + lane < p.groups;
        tiles = there ? max(1, (int)(((uint32_t)(hi - lo) * G + MT - 1) / MT)) : 0;
        keys = there && len >= 0 && len <= longest ? (len + kKeys - 1) / kKeys : 0;
    };
    load(0);
    auto total = [&](auto &&f) {  // over all groups
        int sum = 0;
        for (int c = 0; c < p.groups; c += 64) {
            if (p.groups > 64) load(c);
            sum += __builtin_amdgcn_readlane(wave_sum_up(f()), 63);
        }
        return sum;
    };
    double products = 0.0;
    for (int c = 0; c < p.groups; c += 64) {
        if (p.groups > 64) load(c);
        products += (double)tiles * keys;
    }
    const float work = readlane_f((float)scan_f64(products), 63);
    // Key tiles a part. Parts as if row tiles had no ends are tried first; with the other step they fit for
    // certain (fp32's rounding allowed for), as each row tile may end in a part of less.
    int step = 4;
    auto count = [&]() { return tiles > 0 ? min(most, max(1, (keys + step - 1) / step)) : 0; };
    // (a step of 2^30 is longer than any list: more, from hundreds of thousands of row tiles over long
    // prefixes or from bad offsets, would not be an int)
    auto whole = [](float x) { return (int)fminf(ceilf(x), 0x1p30f); };
    step = max(step, whole(work / (float)items));
    if (total([&]() { return tiles * count(); }) > items) {
        const float spare = (float)max(1, items - total([&]() { return tiles; }));
        step = max(step, whole(work / spare * (1.f + 0x1p-16f)));
    }
    int before = 0, slots = 0;
    for (int c = 0; c < p.groups; c += 64) {
        if (p.groups > 64) load(c);
        const int n = count(), own = tiles * n, end = before + wave_sum_up(own), slot = slots + wave_sum_up(tiles);
        const int at = (int)__popcll(__ballot(c + lane < p.groups && end <= x));
        if (!r.tile.found && at < min(64, p.groups - c)) {
            r.tile.found = true;
            r.tile.b = c + at;
            r.tile.lo = __builtin_amdgcn_readlane(lo, at);
            r.tile.n = __builtin_amdgcn_readlane(hi, at) - r.tile.lo;
            r.tile.slot0 = __builtin_amdgcn_readlane(slot - tiles, at);
            r.tile.per = __builtin_amdgcn_readlane(len, at);
            r.parts = __builtin_amdgcn_readlane(n, at);
            const int i = x - __builtin_amdgcn_readlane(end - own, at), nt = __builtin_amdgcn_readlane(tiles, at);
            r.part = uniform(i / nt);
            r.slot = r.tile.slot0 + i - r.part * nt;
        }
        before = __builtin_amdgcn_readlane(end, 63);
        slots = __builtin_amdgcn_readlane(slot, 63);
    }
    r.tile.ordered = !__any(bad);
    r.tile.found = r.tile.found && r.tile.ordered;
    return r;
}

// A group's prefix: rows of all its sequences, cached keys alone. `b` of the tile is the group.
struct SharedKeys {
    const PrefixArgs &p;
    const Slot &l;
    static constexpr bool kOwnRows = false, kSplit = true;
    __device__ __forceinline__ const WindowArgs &args() const { return p.w; }
    template <int MT>
    __device__ __forceinline__ bool find(int G, int slot, bool, RowTile &t, uint64_t &, int &) const {
        t.b = l.b, t.lo = l.lo, t.n = l.n, t.slot0 = l.slot0, t.len = l.per;
        t.tile = slot - t.slot0;
        if (t.tile * MT >= t.n * G) return false;
        t.i0 = uniform(t.tile * MT / G);
        t.i1 = min(t.n, uniform((t.tile * MT + MT + G - 1) / G));
        t.status = t.len < 0 || t.len > ((int64_t)p.max_prefix_pages << p.w.s.page_shift) || (t.len > 0 && p.w.s.pages == 0)
                       ? BOLE_TREE_BAD_CACHE : BOLE_TREE_OK;
        t.n1 = t.n3 = t.n4 = t.w0 = t.o2 = t.all_from = 0;
        t.n2 = t.len;
        t.own0 = t.total = (t.len + kKeys - 1) & ~(kKeys - 1);
        return true;
    }
    __device__ __forceinline__ const int32_t *table(int g) const { return p.prefix_table + (size_t)g * p.max_prefix_pages; }
    // (each part its own keys' pages: the join asks all of them)
    __device__ __forceinline__ int pages_status(const RowTile &t, int x0, int x1) const {
        return prefix_pages_status(p, t.b, x0, min(x1, t.len));
    }
};

// How a call runs: form, row tiles (slots) and parts of either kind of key list.
struct PrefixPlan {
    bool f32, own_tokens, shared_tokens;
    int own_slots, own_parts, shared_slots, shared_items, shared_parts;
};

struct PrefixParts {
    WindowParts own, shared;
    int own_slots, shared_slots, shared_items, shared_blocks;
};

// An item of the prefixes: its part, and, with the last one, marks where parts of others would be.
template <int MT, class Body>
__device__ __forceinline__ void shared_item(const PrefixArgs &p, const PrefixParts &parts, int block, Body &&body) {
    const WindowShape &s = p.w.s;
    const int x = uniform(block / s.HK), hk = block - x * s.HK, G = s.H / s.HK;
    const Deal d = deal<MT>(p, G, x, parts.shared_items, parts.shared.n);
    if (!d.tile.found) return;
    WindowParts mine = parts.shared;
    mine.n = d.parts;
    if (d.part == d.parts - 1) {
        const int r0 = (d.slot - d.tile.slot0) * MT, rows = min(MT, d.tile.n * G - r0);
        for (int i = threadIdx.x; i < rows * (parts.shared.n - d.parts); i += 256) {
            const int part = i / rows, R = r0 + i - part * rows, row = R / G;
            const size_t at = (size_t)(d.parts + part) * s.T * s.H + (size_t)(d.tile.lo + row) * s.H + hk * G + (R - row * G);
            mine.ml[at * 2] = -INFINITY;
            mine.ml[at * 2 + 1] = 0.f;
        }
    }
    body(SharedKeys{p, d.tile}, mine, d.slot * s.HK + hk, d.part);
}

// The workgroups of the prefixes come first: theirs is the most work.
template <int D, bool OWN_TOKENS, bool SHARED_TOKENS>
__global__ __launch_bounds__(256, 2) void prefix_kernel(const PrefixArgs p, const PrefixParts parts) {
    constexpr int LDS = (OWN_TOKENS && SHARED_TOKENS) ? kTokensLds<D>
                                                      : (kRowsLds<D> > kTokensLds<D> ? kRowsLds<D> : kTokensLds<D>);
    __shared__ __align__(16) char s_mem[LDS];
    const int HK = p.w.s.HK;
    const int bx = blockIdx.x;
    if (bx < parts.shared_blocks) {
        shared_item<SHARED_TOKENS ? kTokenTile : kRowTile>(
            p, parts, bx, [&](const SharedKeys &keys, const WindowParts &mine, int block, int part) {
                if constexpr (SHARED_TOKENS) tokens_body<D>(keys, mine, parts.shared_slots, block, part, s_mem);
                else rows_body<D>(keys, mine, parts.shared_slots, block, part, s_mem);
            });
    } else {
        const int x = bx - parts.shared_blocks, per = parts.own_slots * HK;
        const int part = uniform(x / per), block = x - part * per;
        if constexpr (OWN_TOKENS) tokens_body<D>(OwnKeys{p}, parts.own, parts.own_slots, block, part, s_mem);
        else rows_body<D>(OwnKeys{p}, parts.own, parts.own_slots, block, part, s_mem);
    }
}

template <int D>
__global__ __launch_bounds__(256, 2) void prefix_f32_kernel(const PrefixArgs p, const PrefixParts parts) {
    __shared__ __align__(16) char s_mem[kF32Lds<D>];
    const int HK = p.w.s.HK;
    if ((int)blockIdx.x < parts.shared_blocks) {
        shared_item<kF32Tile>(p, parts, blockIdx.x, [&](const SharedKeys &keys, const WindowParts &mine, int block, int part) {
            f32_body<D>(keys, mine, parts.shared_slots, block, part, s_mem);
        });
    } else {
        const int x = blockIdx.x - parts.shared_blocks, per = parts.own_slots * HK, part = uniform(x / per);
        f32_body<D>(OwnKeys{p}, parts.own, parts.own_slots, x - part * per, part, s_mem);
    }
}

// Joins the parts of a row and head (at most 64), a wavefront each, in a fixed order; a lane has
// D / 64 dimensions (96: two of three lanes' worth). KNOWN: what the first AHEAD parts hold is loaded
// before it is known whether the row is anybody's and which of its parts there are: it only has to be
// there. Otherwise AHEAD at once of those that there are.
template <typename T, int D, int AHEAD, bool KNOWN>
__global__ __launch_bounds__(256) void prefix_join_kernel(const PrefixArgs p, const PrefixParts parts) {
    constexpr int E = D == 64 ? 1 : 2;
    typedef float wide __attribute__((ext_vector_type(E)));
    const WindowArgs &a = p.w;
    const WindowShape &s = a.s;
    const int lane = lane_id(), n_own = parts.own.n, n_all = n_own + parts.shared.n;
    const int64_t at = (int64_t)blockIdx.x * 4 + uniform(threadIdx.x >> 6), all = (int64_t)s.T * s.H;
    const bool line = at < all, has = lane * E < D;
    const float *src = parts.own.o + (line ? at : 0) * D + (has ? lane * E : 0);
    float2 x = {-INFINITY, 0.f};
    wide v[AHEAD];
    if (line) {
        if (lane < n_all) x = *reinterpret_cast<const float2 *>(parts.own.ml + (lane * all + at) * 2);
        if constexpr (KNOWN) {
#pragma unroll
            for (int i = 0; i < AHEAD; ++i) v[i] = *reinterpret_cast<const wide *>(src + min(i, n_all - 1) * all * D);
        }
    }
    const bool ordered = offsets_ordered(a.offsets, s.B, s.T) &&
                         (p.groups == 0 || offsets_ordered(p.group_offsets, p.groups, s.B));
    if (!ordered) {
        if (at == 0 && a.status)
            for (int b = lane; b < s.B; b += 64) a.status[b] = BOLE_TREE_BAD_SIZE;
        return;
    }
    if (!line) return;
    const int row = uniform((int)(at / s.H)), h = (int)(at - (int64_t)row * s.H);
    if (row < a.offsets[0] || row >= a.offsets[s.B]) return;
    int n = n_own;
    if (p.groups > 0 && row >= a.offsets[p.group_offsets[0]] && row < a.offsets[p.group_offsets[p.groups]]) n = n_all;
    const float m = lane < n ? x.x : -INFINITY, l = lane < n ? x.y : 0.f;
    const float own = readlane_f(l, 0);  // (all parts of a bad sequence say the same, of a bad prefix some)
    if (own == kLeftRow) return;
    T *out = static_cast<T *>(a.out) + at * D;
    if (__any(l == kNanRow)) {
        if (own != kNanRow && h == 0 && lane == 0 && a.status) a.status[sequence_of(a.offsets, s.B, row)] = BOLE_TREE_BAD_CACHE;
        for (int e = lane; e < D; e += 64) out[e] = (T)__builtin_nanf("");
        return;
    }
    float top = m;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) top = fmaxf(top, __shfl_xor(top, d, 64));
    const float f = lane < n ? __builtin_amdgcn_exp2f(m - top) : 0.f;
    float sum = f * l;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) sum += __shfl_xor(sum, d, 64);
    wide o = (wide)0.f;
    uint64_t live = __ballot(lane < n && l != 0.f);  // (a part without keys has no sums)
    if constexpr (KNOWN) {
#pragma unroll
        for (int i = 0; i < AHEAD; ++i)
            if ((live >> i) & 1) o += readlane_f(f, i) * v[i];
        live = AHEAD < 64 ? live >> AHEAD << AHEAD : 0;
    }
    while (live) {
        float w[AHEAD];
        int at_part = 0;
#pragma unroll
        for (int i = 0; i < AHEAD; ++i) {
            w[i] = 0.f;
            if (live) at_part = __builtin_ctzll(live), w[i] = readlane_f(f, at_part);
            live &= live - 1;
            v[i] = *reinterpret_cast<const wide *>(src + at_part * all * D);
        }
#pragma unroll
        for (int i = 0; i < AHEAD; ++i) o += w[i] * v[i];
    }
    if (has) {
#pragma unroll
        for (int e = 0; e < E; ++e) out[lane * E + e] = (T)(o[e] / sum);
    }
}

// ---- host

static bool covers(const bole_prefix_dims_t &d) {
    return !(d.flags & BOLE_FLAG_FORCE_GENERIC) &&
           (d.head_dim == 64 || d.head_dim == 96 || d.head_dim == 128) && d.batch > 0;
}

// Parts so that `wanted` workgroups run, no more than one for each 256 keys begun, nor than `most`.
static int parts_for(int64_t workgroups, int64_t keys, int wanted, int most) {
    int64_t n = (wanted + workgroups - 1) / workgroups;
    if (n > (keys + 255) / 256) n = (keys + 255) / 256;
    return (int)(n > most ? most : n < 1 ? 1 : n);
}

// From a call's sizes alone: the tokens form for up to one of its tiles a list on average, as windowed
// attention's rule; of own lists parts so that 512 workgroups run, of prefixes 256, one a CU with the
// own lists' beside them, as a part's sums are written and read again (three batches in turn: 64
// tokens over 16384 50 us, with 384 or 512 workgroups 55 and 61; 128 tokens 77, 86 and 91). Where that is
// three parts or fewer it would leave some CUs two workgroups and others one: 512 (trees of up to 64
// nodes over one prefix of 8192, 24 of them 150 us, with 256 workgroups 157, 48 276 and 303; 64 of up to
// 16 nodes, just past the edge, 140 and 128), or 400 of several prefixes, whose parts are of like length
// (50 trees over four prefixes of up to 8192: 81 us, with 256, 320 and 512 87, 81 and 86; 64 larger ones
// 146, 209, 212 and 146). Of several prefixes one may have three times the average's parts. Lengths
// are not known here: the longest count.
static PrefixPlan plan(const bole_prefix_dims_t &d) {
    PrefixPlan p;
    const int64_t G = d.heads / d.kv_heads, rows = d.total_rows * G;
    p.f32 = d.dtype == BOLE_DTYPE_F32;
    p.own_tokens = !p.f32 && rows <= (int64_t)kTokenTile * d.batch;
    p.shared_tokens = p.own_tokens && rows <= (int64_t)kTokenTile * d.groups;
    const int own = p.f32 ? kF32Tile : p.own_tokens ? kTokenTile : kRowTile;
    const int shared = p.f32 ? kF32Tile : p.shared_tokens ? kTokenTile : kRowTile;
    p.own_slots = (int)(rows / own + d.batch);
    p.own_parts = parts_for((int64_t)p.own_slots * d.kv_heads, (int64_t)d.max_pages * d.page_size + 1, 512, 16);
    p.shared_slots = (int)(d.groups == 1 ? (rows > 0 ? (rows + shared - 1) / shared : 1) : rows / shared + d.groups);
    if (d.groups > 0) {
        const int64_t blocks = (int64_t)p.shared_slots * d.kv_heads, keys = (int64_t)d.max_prefix_pages * d.page_size;
        const int wanted = blocks <= 85 ? 256 : d.groups == 1 ? 512 : 400;
        const int64_t items = wanted / d.kv_heads;  // of a key head
        p.shared_parts = parts_for(d.groups == 1 ? blocks : (blocks + 2) / 3, keys, wanted, 48);
        p.shared_items = (int)(items > p.shared_slots + 1 ? items : p.shared_slots + 1);
        if (d.groups == 1) p.shared_items = p.shared_slots * p.shared_parts;
    } else {
        p.shared_slots = p.shared_items = p.shared_parts = 0;
    }
    return p;
}

size_t prefix_workspace(const bole_prefix_dims_t &d) {
    if (!covers(d)) return 0;
    const PrefixPlan p = plan(d);
    return (size_t)(p.own_parts + p.shared_parts) * d.total_rows * d.heads * (d.head_dim + 2) * sizeof(float);
}

bool prefix_mfma_applies(const bole_prefix_dims_t &d, const PrefixArgs &a) {
    uintptr_t bits = 0;
    for (const void *p : {a.w.q, a.w.k, a.w.v, a.w.k_cache, a.w.v_cache, static_cast<const void *>(a.w.out)})
        bits |= reinterpret_cast<uintptr_t>(p);
    return covers(d) && bits % 16 == 0;
}

template <typename T, int D>
static hipError_t launch_join(const PrefixArgs &a, const PrefixParts &parts, hipStream_t stream) {
    const int64_t lines = (int64_t)a.w.s.T * a.w.s.H;
    const dim3 grid((unsigned)(lines > 0 ? (lines + 3) / 4 : 1)), block(256);
    // Few parts, and all of one prefix's, are there for most rows and loaded ahead; of several prefixes
    // most rows have fewer than the longest's.
    const int n = parts.own.n + parts.shared.n;
    if (n <= 3) prefix_join_kernel<T, D, 3, true><<<grid, block, 0, stream>>>(a, parts);
    else if (n <= 8) prefix_join_kernel<T, D, 8, true><<<grid, block, 0, stream>>>(a, parts);
    else if (a.groups <= 1) prefix_join_kernel<T, D, 16, true><<<grid, block, 0, stream>>>(a, parts);
    else prefix_join_kernel<T, D, 8, false><<<grid, block, 0, stream>>>(a, parts);
    return hipGetLastError();
}

template <int D>
static hipError_t launch_width(const PrefixArgs &a, const PrefixPlan &p, const PrefixParts &parts, hipStream_t stream) {
    const int64_t HK = a.w.s.HK;
    const dim3 block(256), grid((unsigned)(parts.shared_blocks + p.own_slots * HK * p.own_parts));
    if (p.f32) prefix_f32_kernel<D><<<grid, block, 0, stream>>>(a, parts);
    else if (p.own_tokens && p.shared_tokens) prefix_kernel<D, true, true><<<grid, block, 0, stream>>>(a, parts);
    else if (p.own_tokens) prefix_kernel<D, true, false><<<grid, block, 0, stream>>>(a, parts);
    else prefix_kernel<D, false, false><<<grid, block, 0, stream>>>(a, parts);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    return p.f32 ? launch_join<float, D>(a, parts, stream) : launch_join<__bf16, D>(a, parts, stream);
}

hipError_t launch_prefix_mfma(const PrefixArgs &a, const bole_prefix_dims_t &d, void *workspace, hipStream_t stream) {
    const PrefixPlan p = plan(d);
    const size_t lines = (size_t)d.total_rows * d.heads, all = p.own_parts + p.shared_parts;
    float *o = static_cast<float *>(workspace), *ml = o + all * lines * d.head_dim;
    PrefixParts parts;
    parts.own = {o, ml, p.own_parts};
    parts.shared = {o + p.own_parts * lines * d.head_dim, ml + p.own_parts * lines * 2, p.shared_parts};
    parts.own_slots = p.own_slots;
    parts.shared_slots = p.shared_slots;
    parts.shared_items = p.shared_items;
    parts.shared_blocks = p.shared_items * d.kv_heads;
    switch (d.head_dim) {
        case 64: return launch_width<64>(a, p, parts, stream);
        case 96: return launch_width<96>(a, p, parts, stream);
        default: return launch_width<128>(a, p, parts, stream);
    }
}

}  // namespace bole
