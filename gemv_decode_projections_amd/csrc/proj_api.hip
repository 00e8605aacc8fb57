// C ABI of the projection library: layer table, prepare/repack, m-keyed
// dispatch and launch. Declarations and the call contract are in proj.h.
#include <string.h>

#include <algorithm>
#include <vector>

#include <hip/hip_ext.h>

#include "../../include/proj.h"
#include "../../include/proj_bench.h"
#include "repack.h"
#include "rowdot.h"
#include "skinny.h"
#include "tiled.h"
#include "variants.h"
#include "wide.h"

// Split-K scratch of proj_run_noalloc, for callers that cannot allocate: one
// fixed array in the library's device image, so each GPU holds its own copy
// until the process ends. Regions, in order: polled partials (every word all
// ones between launches), counted partials, arrival counters (zero between
// launches). Host code never passes this name to a kernel: it stands for a
// host-side shadow; the device address comes from hipGetSymbolAddress.
constexpr size_t kScratchPolled = 4u << 20;
constexpr size_t kScratchCounted = 16u << 20;
constexpr size_t kScratchCounters = 1u << 14;
constexpr size_t kScratchBytes = kScratchPolled + kScratchCounted + kScratchCounters * sizeof(uint32_t);
static __device__ __align__(256) unsigned char scratch[kScratchBytes];

namespace gdp {

static int g_last_hip = 0;

// Shared with the block operators (block_common.h).
int hip_fail(hipError_t e)
{
    g_last_hip = (int)e;
    return PROJ_ERR_HIP;
}

namespace {

struct LayerInfo {
    const char *name;
    int N;
    int K;
    int w_bytes;   // bytes per weight element
    int o_bytes;   // bytes per output element
};

// Guide ch. 1 "The problem, the judge and the speed of light", §1.1.
constexpr LayerInfo kLayers[PROJ_NUM_LAYERS] = {
    {"qkv_gate", 2304, 8192, 2, 2},
    {"o", 8192, 1024, 2, 2},
    {"pooler", 4096, 8192, 2, 2},
    {"unpooler", 8192, 4096, 2, 2},
    {"router", 256, 8192, 4, 4},
};
constexpr int kSliceMaxM = 8;        // unpooler computes rows 0..1023 at m <= 8
constexpr int kSliceRows = 1024;

// Rows kept in row-major order for the row-dot kernel: the whole router and
// the unpooler's slice (the other layers have enough 16-row blocks to fill
// the chip with the MFMA kernels).
constexpr int kRowMajorRows[PROJ_NUM_LAYERS] = {0, 0, 0, kSliceRows, 256};

constexpr size_t kWsBytes = 32u << 20;       // split-K partials per layer (each of the two workspaces)
constexpr size_t kCounters = 1u << 16;       // split-K arrival counters per layer
// Token counts scanned for the kernels the dispatch table can pick: past this
// count every layer's plan is the same kernel with a larger grid.
constexpr int kPlanScanM = 16384;
// Largest token count: keeps every tile count and rounding in the planning
// arithmetic inside int (x alone would then take 2 TB or more).
constexpr int kMaxM = 1 << 30;
// proj_config.flags bit 4 (skinny kernel, test only): the splits that do not
// reduce drop their partials and the reducer polls once, so every reducer
// gives up; a host-forced stand-in for a split that never arrives.
constexpr int kFlagTestLostSplit = 16;
// proj_config.flags bits 5 / 6 (skinny kernel, one 16-token block): each wave
// loads its activation slice for at most 4 / 8 tokens into registers once.
constexpr int kFlagPreload4 = 32;
constexpr int kFlagPreload8 = 64;
// proj_config.flags bit 7 (wide-tile kernel): activations by LDS DMA.
constexpr int kFlagDma = 128;
// proj_config.flags bit 8 (skinny kernel, rb 1, one token block): the stream
// partition of the (row block, k-step) units over the workgroups.
constexpr int kFlagStream = 256;

struct LayerState {
    void *wp = nullptr;
    f32x4 *ws = nullptr;          // tiled / wide split-K partials (arrival counters)
    uint32_t *counters = nullptr;
    uint64_t *pws = nullptr;      // skinny split-K partials (polled; all ones between launches)
    uint16_t *zrow = nullptr;     // K zero BF16 values: activation rows past m
    void *wrow = nullptr;         // row-major copy of the first wrow_rows rows (row-dot kernel)
    int wrow_rows = 0;
    // 12-bit form (BF16 layers whose rows need at most kZMaxSlots corrections)
    uint32_t *wz = nullptr;       // packed 12-bit fragments
    uint64_t *zexc = nullptr;     // corrections: N rows x zcr slots
    int zcr = -1;                 // slots per row; -1: no 12-bit form
    uint32_t zt0 = 0, zt1 = 0;    // exponent table
    uint32_t *giveups = nullptr;  // polled split-K: reducer give-ups since prepare / last reset
    size_t ws_bytes = kWsBytes;   // capacity of ws
    size_t pws_bytes = kWsBytes;  // capacity of pws
    size_t n_counters = kCounters;
    int device = -1;
    bool prepared = false;
};

LayerState g_layers[PROJ_NUM_LAYERS];

// Device address of `scratch` on each GPU (set once per device by prepare).
constexpr int kMaxDevices = 64;
void *g_scratch[kMaxDevices] = {};


bool aligned16(const void *p) { return ((uintptr_t)p & 15u) == 0; }

int n_eff_of(int layer, int m)
{
    if (layer == PROJ_UNPOOLER && m <= kSliceMaxM)
        return kSliceRows;
    return kLayers[layer].N;
}

constexpr int kSkinnyPartCount = 5;
const SkinnyVariant *const kSkinnyParts[kSkinnyPartCount] = {kSkinnyPartBf16Nt1, kSkinnyPartBf16Nt2, kSkinnyPartF32,
                                                             kSkinnyPartZ, kSkinnyPartStream};

int skinny_part_count(int p)
{
    const int counts[kSkinnyPartCount] = {kSkinnyPartBf16Nt1Count, kSkinnyPartBf16Nt2Count, kSkinnyPartF32Count,
                                          kSkinnyPartZCount, kSkinnyPartStreamCount};
    return counts[p];
}

const SkinnyVariant *find_variant(int nt, int rb, int waves, int spw, int f32w, int z, int xp, int skm)
{
    for (int p = 0; p < kSkinnyPartCount; ++p)
        for (int i = 0; i < skinny_part_count(p); ++i) {
            const SkinnyVariant &v = kSkinnyParts[p][i];
            if (v.nt == nt && v.rb == rb && v.waves == waves && v.spw == spw && v.f32w == f32w && v.z == z &&
                v.xp == xp && v.skm == skm)
                return &v;
        }
    return nullptr;
}

const TiledVariant *find_tiled(int bmb, int bnb, int waves, int depth, int f32w)
{
    for (int i = 0; i < kTiledVariantCount; ++i) {
        const TiledVariant &v = kTiledVariants[i];
        if (v.bmb == bmb && v.bnb == bnb && v.wr * v.kg == waves && v.depth == depth && v.f32w == f32w)
            return &v;
    }
    return nullptr;
}

int wide_variant_count() { return kWideVariantCount + kWideDmaVariantCount; }

const WideVariant &wide_variant_at(int i)
{
    return i < kWideVariantCount ? kWideVariants[i] : kWideDmaVariants[i - kWideVariantCount];
}

const WideVariant *find_wide(int bmb, int bnb, int depth, int f32w, int waves, int xdma)
{
    for (int i = 0; i < wide_variant_count(); ++i) {
        const WideVariant &v = wide_variant_at(i);
        if (v.bmb == bmb && v.bnb == bnb && v.depth == depth && v.f32w == f32w && v.waves == waves &&
            v.xdma == xdma)
            return &v;
    }
    return nullptr;
}

const RowVariant *find_row(int mcap, int r, int kit, int f32w)
{
    for (int i = 0; i < kRowVariantCount; ++i) {
        const RowVariant &v = kRowVariants[i];
        if (v.mcap == mcap && v.r == r && v.kit == kit && v.f32w == f32w)
            return &v;
    }
    return nullptr;
}

int skinny_variants()
{
    int n = 0;
    for (int p = 0; p < kSkinnyPartCount; ++p)
        n += skinny_part_count(p);
    return n;
}

int total_variants() { return skinny_variants() + kTiledVariantCount + kRowVariantCount + wide_variant_count(); }

const SkinnyVariant *variant_at(int i)
{
    if (i < 0)
        return nullptr;
    for (int p = 0; p < kSkinnyPartCount; ++p) {
        if (i < skinny_part_count(p))
            return &kSkinnyParts[p][i];
        i -= skinny_part_count(p);
    }
    return nullptr;
}

// Resolved launch of one configuration (only the argument block of its kind is used).
struct Launch {
    const void *fn;
    int kind;
    SkinnyArgs sargs;
    TiledArgs targs;
    RowArgs rargs;
    WideArgs wargs;
    int grid;
    int block;
};

// Checks that `c` tiles (layer, m) exactly and fits the workspace of layer
// state `st`; fills `L`.
int resolve(int layer, int m, const proj_config &c, Launch &L, const LayerState &st)
{
    const LayerInfo &li = kLayers[layer];
    const int f32w = li.w_bytes == 4 ? 1 : 0;
    const int KS = li.K / kStepK;
    const int ne = n_eff_of(layer, m);
    if (c.ksplit < 1)
        return PROJ_ERR_UNSUPPORTED;
    // Flag bits each kind understands: 0 placement (all), 2 12-bit weights
    // (kind 0), 3 stream mode (kind 3), 4 the test-only lost split (kind 0),
    // 5 / 6 preloaded activations (kind 0), 7 activations by LDS DMA (kind 3),
    // 8 the stream partition (kind 0).
    const int known = 1 | (c.kind == 0 ? 4 | kFlagTestLostSplit | kFlagPreload4 | kFlagPreload8 | kFlagStream : 0) |
                      (c.kind == 3 ? 8 | kFlagDma : 0);
    if (c.flags & ~known)
        return PROJ_ERR_UNSUPPORTED;
    if (c.kind == 0) {
        const int z = (c.flags & 4) ? 1 : 0;
        if (z && st.zcr < 0)
            return PROJ_ERR_UNSUPPORTED;              // no 12-bit form for this layer
        const int pre = c.flags & (kFlagPreload4 | kFlagPreload8);
        const int xp = pre == kFlagPreload4 ? 4 : pre == kFlagPreload8 ? 8 : 0;
        if (pre && (!xp || m > xp))
            return PROJ_ERR_UNSUPPORTED;              // both bits, or more tokens than the preload holds
        const int skm = (c.flags & kFlagStream) ? 1 : 0;
        const SkinnyVariant *v = find_variant(c.nt, c.rb, c.waves, c.spw, f32w, z, xp, skm);
        if (!v)
            return PROJ_ERR_UNSUPPORTED;
        if (skm) {
            // Units: (16-row block, k-step) pairs, dealt in shares of
            // waves * spw; one token block; every row block covered by at
            // most kSkMaxParts shares (bounded by ceil(KS / P) + 1).
            const long long P = (long long)c.waves * c.spw;
            const long long units = (long long)(ne / kRowsPerBlock) * KS;
            if (xp || c.rb != 1 || c.ksplit != 1 || ne % kRowsPerBlock != 0 || m > 16 * c.nt || units % P != 0 ||
                P > KS)                                // a share spans at most two row blocks
                return PROJ_ERR_UNSUPPORTED;
            if ((KS + P - 1) / P + 1 > kSkMaxParts)
                return PROJ_ERR_UNSUPPORTED;
            if ((long long)(ne / kRowsPerBlock) * kSkMaxParts * c.nt * kWave * (long long)sizeof(f32x4) >
                (long long)st.pws_bytes)
                return PROJ_ERR_UNSUPPORTED;
            const long long grid = units / P;
            L.fn = v->fn;
            L.kind = 0;
            L.grid = (int)grid;
            L.block = (c.waves + z) * kWave;
            SkinnyArgs &A = L.sargs;
            A.wz = st.wz;
            A.wz_bytes = (uint32_t)((size_t)li.N * li.K * 3 / 2);
            A.zt0 = st.zt0;
            A.zt1 = st.zt1;
            A.zcr = z ? st.zcr : 0;
            A.zexc = st.zexc;
            A.wp = st.wp;
            A.pws = st.pws;
            A.m = m;
            A.K = li.K;
            A.n_eff = ne;
            A.n_rt = (int)grid;
            A.n_tt = 1;
            A.ksplit = 1;
            A.xcd_remap = (!(c.flags & 1) && grid % 8 == 0) ? 1 : 0;
            A.giveups = st.giveups;
            A.drop_publish = (c.flags & kFlagTestLostSplit) ? 1 : 0;
            A.poll_limit = A.drop_publish ? 1 : kPollLimit;
            return PROJ_OK;
        }
        if (c.waves * c.spw * c.ksplit != KS)
            return PROJ_ERR_UNSUPPORTED;
        if (ne % (kRowsPerBlock * c.rb) != 0)
            return PROJ_ERR_UNSUPPORTED;
        const int n_rt = ne / (kRowsPerBlock * c.rb);
        const int n_tt = (m + 16 * c.nt - 1) / (16 * c.nt);
        const long long grid = (long long)n_rt * n_tt * c.ksplit;
        if (grid < 1 || grid > 0x7fffffffLL)
            return PROJ_ERR_UNSUPPORTED;
        if (c.ksplit > 1) {
            const long long elems = (long long)c.rb * c.nt * kWave;
            if ((long long)n_rt * n_tt * c.ksplit * elems * (long long)sizeof(f32x4) > (long long)st.pws_bytes)
                return PROJ_ERR_UNSUPPORTED;
        }
        L.fn = v->fn;
        L.kind = 0;
        L.grid = (int)grid;
        L.block = (c.waves + z) * kWave;
        SkinnyArgs &A = L.sargs;
        A.wz = st.wz;
        A.wz_bytes = (uint32_t)((size_t)li.N * li.K * 3 / 2);
        A.zt0 = st.zt0;
        A.zt1 = st.zt1;
        A.zcr = z ? st.zcr : 0;
        A.zexc = st.zexc;
        A.wp = st.wp;
        A.pws = st.pws;
        A.m = m;
        A.K = li.K;
        A.n_eff = ne;
        A.n_rt = n_rt;
        A.n_tt = n_tt;
        A.ksplit = c.ksplit;
        A.xcd_remap = (!(c.flags & 1) && grid % 8 == 0) ? 1 : 0;
        A.giveups = st.giveups;
        A.drop_publish = (c.flags & kFlagTestLostSplit) ? 1 : 0;
        A.poll_limit = A.drop_publish ? 1 : kPollLimit;
        return PROJ_OK;
    }
    if (c.kind == 1) {
        // rb = 16-row blocks per tile, nt = 16-token blocks per tile,
        // spw = prefetch depth in super-steps (kg k-steps each)
        const TiledVariant *v = find_tiled(c.rb, c.nt, c.waves, c.spw, f32w);
        if (!v)
            return PROJ_ERR_UNSUPPORTED;
        if (KS % (c.spw * c.ksplit * v->kg) != 0)   // k-steps per workgroup: a multiple of kg * depth
            return PROJ_ERR_UNSUPPORTED;
        if (ne % (kRowsPerBlock * c.rb) != 0)
            return PROJ_ERR_UNSUPPORTED;
        const int n_rt = ne / (kRowsPerBlock * c.rb);
        const int n_tt = (m + 16 * c.nt - 1) / (16 * c.nt);
        const long long grid = (long long)n_rt * n_tt * c.ksplit;
        if (grid < 1 || grid > 0x7fffffffLL)
            return PROJ_ERR_UNSUPPORTED;
        if (c.ksplit > 1) {
            const long long tile_bytes = (long long)c.rb * c.nt * kWave * 16;
            if ((long long)n_rt * n_tt * c.ksplit * tile_bytes > (long long)st.ws_bytes)
                return PROJ_ERR_UNSUPPORTED;
            if ((long long)n_rt * n_tt > (long long)st.n_counters)
                return PROJ_ERR_UNSUPPORTED;
        }
        L.fn = v->fn;
        L.kind = 1;
        L.grid = (int)grid;
        L.block = c.waves * kWave;
        TiledArgs &A = L.targs;
        A.wp = st.wp;
        A.zrow = st.zrow;
        A.ws = reinterpret_cast<float *>(st.ws);
        A.counters = st.counters;
        A.m = m;
        A.K = li.K;
        A.n_eff = ne;
        A.n_rt = n_rt;
        A.n_tt = n_tt;
        A.ksplit = c.ksplit;
        A.xcd_remap = (!(c.flags & 1) && grid % 8 == 0) ? 1 : 0;
        return PROJ_OK;
    }
    if (c.kind == 3) {
        // rb = 16-row blocks per tile (waves x rb/waves, 4 or 8 waves), nt = 16-token blocks,
        // spw = weight prefetch depth in k-steps; K split unevenly in
        // super-steps of 2 (4 at depth 16) k-steps. flags bit 3: stream mode,
        // ksplit = number of workgroups sharing all tiles' super-steps.
        const WideVariant *v = find_wide(c.rb, c.nt, c.spw, f32w, c.waves, (c.flags & kFlagDma) ? 1 : 0);
        if (!v)
            return PROJ_ERR_UNSUPPORTED;
        if (ne % (kRowsPerBlock * c.rb) != 0 || c.ksplit < 1)
            return PROJ_ERR_UNSUPPORTED;
        const int nss = KS / wide_superstep(c.spw);
        const int n_rt = ne / (kRowsPerBlock * c.rb);
        const int n_tt = (m + 16 * c.nt - 1) / (16 * c.nt);
        const long long tiles = (long long)n_rt * n_tt;
        const bool stream = (c.flags & 8) != 0;
        long long grid = 0;
        int slots = c.ksplit;                          // workspace slots per tile
        if (!stream) {
            if (c.ksplit > nss)
                return PROJ_ERR_UNSUPPORTED;
            grid = tiles * c.ksplit;
        } else {
            // Every share non-empty (G <= tiles * nss); slots = the most
            // workgroups any tile is shared by.
            const long long I = tiles * nss;
            const long long G = c.ksplit;
            if (G > I || G > 0x7fffffffLL)
                return PROJ_ERR_UNSUPPORTED;
            auto owner = [&](long long q) { return ((q + 1) * G + I - 1) / I - 1; };
            slots = 1;
            for (long long t = 0; t < tiles; ++t)
                slots = std::max(slots, (int)(owner(t * nss + nss - 1) - owner(t * nss) + 1));
            grid = G;
        }
        if (grid < 1 || grid > 0x7fffffffLL)
            return PROJ_ERR_UNSUPPORTED;
        if (slots > 1) {
            const long long tile_bytes = (long long)c.rb * c.nt * kWave * 16;
            if (tiles * slots * tile_bytes > (long long)st.ws_bytes)
                return PROJ_ERR_UNSUPPORTED;
            if (tiles > (long long)st.n_counters)
                return PROJ_ERR_UNSUPPORTED;
        }
        L.fn = stream ? v->fn_stream : v->fn;
        L.kind = 3;
        L.grid = (int)grid;
        L.block = c.waves * kWave;
        WideArgs &A = L.wargs;
        A.wp = st.wp;
        A.zrow = st.zrow;
        A.ws = reinterpret_cast<float *>(st.ws);
        A.ws_bytes = (uint32_t)st.ws_bytes;
        A.counters = st.counters;
        A.m = m;
        A.K = li.K;
        A.n_eff = ne;
        A.n_rt = n_rt;
        A.n_tt = n_tt;
        A.ksplit = c.ksplit;
        A.xcd_remap = (!(c.flags & 1) && grid % 8 == 0) ? 1 : 0;
        A.maxc = slots;
        return PROJ_OK;
    }
    if (c.kind == 2) {
        // nt = token capacity, rb = rows per workgroup, spw = 2048-wide k chunks per row
        const RowVariant *v = find_row(c.nt, c.rb, c.spw, f32w);
        if (!v || c.waves != kRowWaves || c.ksplit != 1)
            return PROJ_ERR_UNSUPPORTED;
        if (m > c.nt || ne > kRowMajorRows[layer] || ne % c.rb != 0)
            return PROJ_ERR_UNSUPPORTED;
        if (li.K != c.spw * kRowThreads * 8)
            return PROJ_ERR_UNSUPPORTED;
        L.fn = v->fn;
        L.kind = 2;
        L.grid = ne / c.rb;
        L.block = kRowThreads;
        RowArgs &A = L.rargs;
        A.w = st.wrow;
        A.m = m;
        A.K = li.K;
        A.n_eff = ne;
        return PROJ_OK;
    }
    return PROJ_ERR_UNSUPPORTED;
}

// The m-keyed dispatch table. Shapes only: (layer, m) -> configuration.
// Buckets: m <= 8 (one 16-token tile, unpooler slice), 9..16, 17..32 (two
// 16-token tiles), and m > 32. Entries are the fastest measured cold-cache
// configurations on MI355X (kernel duration, plain weight loads).
proj_config plan_default(int layer, int m, int zcr)
{
    struct Entry {
        int nt, rb, waves, spw, ksplit, z;   // z: read the 12-bit weights when the layer has them
        int mode;                            // 1: preloaded activations (bucket 0); 2: stream partition
    };
    // [layer][bucket]: bucket 0: m <= 8, 1: m <= 16, 2: m <= 32. Entries
    // are the fastest of every compiled configuration in cold sweeps (a plain
    // 1 GiB read before each call, so no weight byte is left in L2 or the
    // Infinity Cache), kept where they beat the next one by more than the
    // sweep's noise. The 12-bit form pays wherever the weight stream is long
    // (qkv_gate and pooler to 16 tokens, the full unpooler to 32); o's short
    // stream does not hide the correction wave. Bucket 2 of qkv_gate and the
    // pooler (64-row tiles over both token blocks, a 4-way K split) is not
    // reached: the wide-tile rule below takes them at 17-32 tokens.
    // Up to 8 tokens qkv_gate and the unpooler slice preload each wave's
    // activations (flags bit 5 / 6): A/B 1.5 / 1.0 / 0.7 us faster on
    // qkv_gate at 1 / 4 / 8 tokens, 0.1-0.2 on the slice; no gain on the
    // pooler, which already runs at the plain read floor there. At 9-15
    // tokens qkv_gate runs the stream partition (flags bit 8: its 144 row
    // blocks x 256 k-steps dealt to 256 workgroups of 4 waves x 36 k-steps;
    // A/B against the 4-way split below at m = 9 / 12 / 14 / 16: -0.18 /
    // -0.44 / -0.48 / -0.64 us in one run, +0.06 / -0.10 / - / -0.32 in
    // another) and the unpooler 4-wave workgroups of two row blocks over the
    // whole K (A/B at m = 9 / 12 / 16: 0.24 / 0.28 / 0.20 us faster).
    static const Entry table[PROJ_NUM_LAYERS][3] = {
        /* qkv_gate  144 row blocks, 256 k-steps */
        {{1, 1, 8, 32, 1, 1, 1}, {1, 1, 4, 36, 1, 1, 2}, {2, 4, 8, 8, 4, 0, 0}},
        /* o         512 row blocks,  32 k-steps */
        {{1, 2, 8, 4, 1, 0, 0}, {1, 2, 8, 4, 1, 0, 0}, {2, 2, 4, 8, 1, 0, 0}},
        /* pooler    256 row blocks, 256 k-steps */
        {{1, 1, 8, 32, 1, 1, 0}, {1, 1, 8, 32, 1, 1, 0}, {2, 4, 8, 8, 4, 0, 0}},
        /* unpooler  64 (slice) / 512 row blocks, 128 k-steps */
        {{1, 1, 4, 8, 4, 0, 1}, {1, 2, 4, 32, 1, 1, 0}, {2, 2, 4, 32, 1, 1, 0}},
        /* router    16 row blocks, 256 k-steps of FP32 weights */
        {{1, 1, 8, 4, 8, 0, 0}, {1, 1, 16, 2, 8, 0, 0}, {1, 1, 16, 2, 8, 0, 0}},
    };
    proj_config c{};
    // Few tokens on the router (m <= 8) and the unpooler slice (m <= 4):
    // whole rows per workgroup (row-dot kernel), token capacity rounded up to
    // a power of two. Past 4 tokens the unpooler slice re-reads too much
    // activation data per row and the skinny kernel is faster.
    if ((layer == PROJ_ROUTER && m <= 8) || (layer == PROJ_UNPOOLER && m <= 4)) {
        c.kind = 2;
        c.nt = m <= 1 ? 1 : m <= 2 ? 2 : m <= 4 ? 4 : 8;
        c.rb = layer == PROJ_ROUTER ? 1 : (m <= 2 ? 2 : 4);
        c.waves = kRowWaves;
        c.spw = kLayers[layer].K / (kRowThreads * 8);
        c.ksplit = 1;
        return c;
    }
    c.kind = 0;
    // The pooler at 14-16 tokens on its 12-bit weights: two-row-block 4-wave
    // workgroups with a 2-way split (A/B at m = 14 / 15 / 16: 0.36 / 0.46 /
    // 0.70 us faster than the table's entry; a tie at 12-13, a loss at 9).
    if (layer == PROJ_POOLER && m >= 14 && m <= 16 && zcr >= 0) {
        c.nt = 1;
        c.rb = 2;
        c.waves = 4;
        c.spw = 32;
        c.ksplit = 2;
        c.flags = 4;
        return c;
    }
    // qkv_gate at 16-32 tokens and the pooler at 17-32 on the wide-tile
    // kernel (kind 3): 64-row tiles of 16 tokens (m = 16) or 32 tokens, the
    // activations staged once per workgroup in LDS instead of loaded by every
    // wave, an arrival-counted K split. In-process cold A/B against the
    // skinny plans (us): qkv_gate m = 16 / 17 / 24 / 32 11.88 / 13.76 /
    // 14.62 / 15.62 -> 11.66 / 12.26 / 12.32 / 12.48 (the stream partition
    // stays ahead at 9-13 tokens, a tie at 14); pooler m = 17 / 24 / 28 / 32
    // 17.12 / 17.20 / 17.38 / 17.74 -> 16.86 / 16.76 / 16.92 / 16.84 (within
    // noise at 20). The unpooler (29-32) and o measured no gain.
    if ((layer == PROJ_QKV_GATE && m >= 16 && m <= 32) || (layer == PROJ_POOLER && m >= 17 && m <= 32)) {
        const bool qkv = layer == PROJ_QKV_GATE;
        c.kind = 3;
        c.nt = m <= 16 ? 1 : 2;
        c.rb = 4;
        c.waves = 4;
        c.spw = qkv ? 16 : 8;
        c.ksplit = qkv ? 6 : 4;
        c.flags = qkv ? 0 : kFlagDma;
        return c;
    }
    if (m <= 32) {
        const Entry &e = table[layer][m <= 8 ? 0 : (m <= 16 ? 1 : 2)];
        c.nt = e.nt;
        c.rb = e.rb;
        c.waves = e.waves;
        c.spw = e.spw;
        c.ksplit = e.ksplit;
        c.flags = (e.z && zcr >= 0) ? 4 : 0;
        if (e.mode == 1)
            c.flags |= m <= 4 ? kFlagPreload4 : kFlagPreload8;
        if (e.mode == 2)
            c.flags |= kFlagStream;
        return c;
    }
    // The router at 33-256 tokens stays on the skinny kernel: with 16 row
    // blocks the tiled kernels' 64-row tiles leave most compute units idle
    // or need deep K splits (measured 12-15 us against 8-13.5 here). Two
    // 16-token blocks per workgroup from 65 tokens, two row blocks from 129.
    // Past 256 tokens: the wide-tile kernel's FP32-weight tiles (64 rows x 64
    // tokens, 128 past 1024 tokens; the exact three-part split as in the
    // skinny kernel), K split over up to 8 workgroups, the grid filled to 512
    // (64-token tiles) or 256 workgroups. In-process cold A/B against the
    // skinny plans (us): m = 512 / 896 / 1500 / 2048 / 4096 / 8192 21.8 /
    // 32.6 / 49.9 / 63.8 / 118.2 / 231.5 -> 20.3 / 25.0 / 32.9 / 39.6 / 68.1
    // / 126.3 (a tie at 257-300).
    if (layer == PROJ_ROUTER && m > 256) {
        const int nt = m <= 1024 ? 4 : 8;
        const long tiles = (long)(kLayers[layer].N / 64) * ((m + 16 * nt - 1) / (16 * nt));
        c.kind = 3;
        c.nt = nt;
        c.rb = 4;
        c.waves = 4;
        c.spw = 4;
        int ks = (int)std::max(1L, std::min(8L, (nt == 4 ? 512 : 256) / tiles));
        while (ks > 1 && tiles * ks * c.rb * c.nt * 1024 > (long)kWsBytes)
            --ks;
        c.ksplit = ks;
        c.flags = 0;
        return c;
    }
    if (layer == PROJ_ROUTER) {
        static const Entry rtable[3] = {{1, 1, 16, 4, 4, 0}, {2, 1, 16, 4, 4, 0}, {2, 2, 16, 4, 4, 0}};
        const Entry &e = rtable[m <= 64 ? 0 : m <= 128 ? 1 : 2];
        c.nt = e.nt;
        c.rb = e.rb;
        c.waves = e.waves;
        c.spw = e.spw;
        c.ksplit = e.ksplit;
        return c;
    }
    // (qkv_gate at 33-48 tokens once ran the 12-bit skinny kernel over
    // 16-token tiles; with the weights really cold the wide tiles below are
    // faster: m = 33 / 40 / 48 16.5 / 16.6 / 16.8 -> 14.1 / 14.2 / 14.4 us.)
    // Larger m: the tiled kernel (kind 1) or the wide-tile kernel (kind 3),
    // picked per layer from measured cold-cache sweeps. Buckets: m <= 64,
    // m <= 128, m <= 256 (past 256 tokens the rule further down). Entries:
    // kind, 16-row blocks per tile (rb), 16-token blocks (nt), weight
    // prefetch depth in k-steps, K split; the split shrinks until the partials
    // fit the workspace. A split of 0 means: as many splits (at most 4) as keep the
    // grid within one workgroup per compute unit (a grid past 256 measured
    // far slower: qkv_gate m = 130 with 64-token tiles took 18.7 us at 4
    // splits, 216 workgroups, 32.4 at 5, 270 workgroups, and 24.5 at 3).
    // dma: the wide-tile kernel moves activations by LDS DMA (flags bit 7).
    // In-process cold A/B against register staging (us): pooler m = 128 /
    // 256 / 512 / 1000 24.8 / 32.9 / 53.9 / 88.9 -> 24.3 / 31.6 / 52.5 / 85.3;
    // unpooler m = 256 / 512 / 1000 30.7 / 47.7 / 62.5 -> 30.0 / 47.0 / 60.3;
    // qkv_gate m = 256 25.7 -> 25.1. Elsewhere it tied or lost (qkv_gate
    // m = 128 19.0 -> 19.5; o m = 256 11.3 -> 12.3 at prefetch depth 4). o at
    // 129-256 tokens with depth 8 and DMA, against depth 4 without: m = 160 /
    // 200 / 256 10.56 / 10.74 / 11.08 -> 9.80 / 9.90 / 10.40.
    struct TEntry {
        int kind, rb, nt, waves, depth, ksplit, dma;
    };
    // Measured in the same cold sweeps (m = 64, 128, 256).
    static const TEntry ttable[PROJ_ROUTER][3] = {   // the four BF16 layers
        /* qkv_gate */ {{3, 4, 4, 4, 16, 6, 0}, {3, 4, 4, 4, 16, 3, 0}, {3, 8, 4, 4, 16, 0, 1}},
        /* o        */ {{1, 4, 2, 4, 16, 1, 0}, {1, 8, 2, 4, 8, 1, 0}, {3, 8, 4, 4, 8, 0, 1}},
        /* pooler   */ {{3, 4, 4, 4, 8, 4, 0}, {3, 8, 4, 4, 8, 4, 1}, {3, 8, 8, 8, 8, 0, 1}},
        /* unpooler */ {{1, 4, 2, 4, 16, 1, 0}, {3, 4, 4, 4, 16, 1, 0}, {3, 8, 4, 4, 16, 0, 1}},
    };
    const int ne = n_eff_of(layer, m);
    // The pooler at 129-192 tokens: 256 x 64 tiles on 8 waves with 5 splits
    // (240 workgroups) beat its 128 x 64 tiles with 2 (m = 130 / 160 / 192:
    // 24.6 / 24.9 / 25.6 -> 23.6 / 24.2 / 24.3 us); the other layers, and the
    // pooler at 193-256, measured no gain. A 16-k-step weight prefetch (four
    // k-steps per activation super-step, one barrier per four k-steps) beat
    // depth 8 on this tile: m = 130 / 144 / 160 / 176 / 192 30.00 / 30.00 /
    // 30.48 / 30.70 / 30.94 -> 29.40 / 29.54 / 30.00 / 30.30 / 30.52 us.
    // The unpooler at 129-256 tokens: its 64-token tiles without a split
    // take longer the fuller their last tile, 128 x 128 tiles with 2 splits
    // (256 workgroups) stay near 28.5 us, so the latter once the last
    // 64-token tile holds more than 32 tokens (cold A/B, plan -> 128 x 128,
    // us: m = 168 / 176 / 184 / 192 28.98 / 29.42 / 29.48 / 29.68 -> 28.40
    // / 28.56 / 28.58 / 28.48; m = 232 / 240 / 248 / 256 29.08 / 29.24 /
    // 29.72 / 29.52 -> 28.36 / 28.44 / 28.64 / 29.00; with fewer in the
    // last tile a tie or a loss: m = 136 / 200 / 208 +0.62 / +0.36 / +0.18).
    if (layer == PROJ_UNPOOLER && m > 128 && m <= 256 && (m - 1) % 64 >= 32) {
        c.kind = 3;
        c.rb = 8;
        c.nt = 8;
        c.waves = 4;
        c.spw = 8;
        c.ksplit = 2;
        c.flags = kFlagDma;
        return c;
    }
    if (layer == PROJ_POOLER && m > 128 && m <= 192) {
        c.kind = 3;
        c.rb = 16;
        c.nt = 4;
        c.waves = 8;
        c.spw = 16;
        c.ksplit = 5;
        c.flags = kFlagDma;
        return c;
    }
    // Past 256 tokens: 128 x 128 tiles on 4 waves while that fills the chip
    // with at most 4 K splits (qkv_gate to 896 tokens, the other layers to
    // 512), then 256 x 128 tiles on 8 waves (two per SIMD); the split count
    // the largest that keeps the grid within 256 workgroups (the unpooler and
    // o: no split), activations by LDS DMA where it measured faster; the
    // pooler at 257-320 tokens on 256 x 64 tiles with 3 splits (3.7 us ahead
    // of the 128 x 128 ones there). In-process cold A/B against the earlier
    // rule (256 x 64 tiles on 8 waves while they gave 160 workgroups, else
    // 256 x 128 within 512 workgroups, 256 for o, else 4-wave tiles; tuned
    // with the non-temporal flush), us: qkv_gate m = 300 / 512 / 768 / 1500
    // 33.7 / 40.6 / 53.8 / 87.5 -> 28.3 / 34.0 / 44.4 / 69.2; pooler m = 384 /
    // 512 / 640 / 1000 51.2 / 51.7 / 82.0 / 85.4 -> 42.3 / 44.4 / 53.5 / 71.8;
    // unpooler m = 300 / 512 44.4 / 47.0 -> 39.5 / 41.4; o m = 300 / 512 /
    // 2048 14.7 / 15.9 / 55.5 -> 13.2 / 14.4 / 42.9; ties on the unpooler from
    // 640 tokens up to 2048. Past 2048 tokens (cold sweep, m = 8192) o /
    // unpooler / pooler / qkv_gate 227 / 653 / 608 / 372 -> 167 / 486 / 445 /
    // 309 us, and equal where the earlier rule already chose these tiles.
    if (m > 256) {
        if (layer == PROJ_POOLER && m <= 320) {
            c.kind = 3;
            c.rb = 16;
            c.nt = 4;
            c.waves = 8;
            c.spw = 8;
            c.ksplit = 3;
            c.flags = kFlagDma;
            return c;
        }
        struct Big {
            int maxA, ksmax, dmaA, dmaB;      // last m on 128 x 128 tiles; split cap; DMA per family
        };
        static const Big big[PROJ_ROUTER] = {
            /* qkv_gate */ {896, 4, 0, 0},
            /* o        */ {512, 1, 1, 0},
            /* pooler   */ {512, 4, 1, 1},
            /* unpooler */ {512, 1, 1, 1},
        };
        const Big &b = big[layer];
        const bool A = m <= b.maxA;
        c.kind = 3;
        c.nt = 8;
        c.rb = A ? 8 : 16;
        c.waves = A ? 4 : 8;
        c.spw = 8;
        const long tiles = (long)(ne / (16 * c.rb)) * ((m + 127) / 128);
        int ks = (int)std::max(1L, std::min((long)b.ksmax, 256 / tiles));
        while (ks > 1 && tiles * ks * c.rb * c.nt * 1024 > (long)kWsBytes)
            --ks;
        c.ksplit = ks;
        c.flags = (A ? b.dmaA : b.dmaB) ? kFlagDma : 0;
        return c;
    }
    const TEntry &e = ttable[layer][m <= 64 ? 0 : (m <= 128 ? 1 : 2)];
    c.kind = e.kind;
    c.rb = e.rb;
    c.nt = e.nt;
    c.waves = e.waves;
    c.spw = e.depth;
    const long tiles = (long)(ne / (16 * c.rb)) * ((m + 16 * c.nt - 1) / (16 * c.nt));
    int ks = e.ksplit > 0 ? e.ksplit : (int)std::max(1L, std::min(4L, 256 / tiles));
    while (ks > 1 && tiles * ks * c.rb * c.nt * 1024 > (long)kWsBytes)
        ks = e.kind == 3 ? ks - 1 : ks / 2;   // the tiled kernel splits K into equal powers of two
    c.ksplit = ks;
    c.flags = (e.kind == 3 && e.dma) ? kFlagDma : 0;
    return c;
}

int check_layer(int layer) { return (layer < 0 || layer >= PROJ_NUM_LAYERS) ? PROJ_ERR_LAYER : PROJ_OK; }

int check_run_args(int layer, const void *x, int m, void *out)
{
    if (check_layer(layer))
        return PROJ_ERR_LAYER;
    if (m < 1 || m > kMaxM)
        return PROJ_ERR_M;
    if (!x || !out)
        return PROJ_ERR_NULL;
    if (!aligned16(x) || !aligned16(out))
        return PROJ_ERR_ALIGN;
    const LayerState &st = g_layers[layer];
    if (!st.prepared)
        return PROJ_ERR_NOT_PREPARED;
    int dev = -1;
    hipError_t e = hipGetDevice(&dev);
    if (e != hipSuccess)
        return hip_fail(e);
    if (dev != st.device)
        return PROJ_ERR_DEVICE;
    return PROJ_OK;
}

int launch(const Launch &L, const void *x, void *out, hipStream_t stream, hipEvent_t ev_start = nullptr,
           hipEvent_t ev_stop = nullptr)
{
    SkinnyArgs sargs = L.sargs;
    TiledArgs targs = L.targs;
    RowArgs rargs = L.rargs;
    WideArgs wargs = L.wargs;
    sargs.x = targs.x = rargs.x = wargs.x = static_cast<const uint16_t *>(x);
    sargs.out = targs.out = rargs.out = wargs.out = out;
    void *params[1];
    params[0] = L.kind == 0   ? static_cast<void *>(&sargs)
                : L.kind == 1 ? static_cast<void *>(&targs)
                : L.kind == 3 ? static_cast<void *>(&wargs)
                              : static_cast<void *>(&rargs);
    hipError_t e;
    if (ev_start || ev_stop)
        e = hipExtLaunchKernel(L.fn, dim3(L.grid), dim3(L.block), params, 0, stream, ev_start, ev_stop, 0);
    else
        e = hipLaunchKernel(L.fn, dim3(L.grid), dim3(L.block), params, 0, stream);
    if (e != hipSuccess)
        return hip_fail(e);
    return PROJ_OK;
}

// The 12-bit form of a BF16 layer (format: common.h decode12, repack.h
// repack_z_kernel). The exponent table is the eight consecutive values of
// BF16 bits 14..8 that cover the most weights (the report's round-5 rule);
// every other weight gets a correction slot in its row: k, its own bits w
// and the bits d that its clamped 12-bit code decodes to. Rows are padded to
// the largest count with empty slots (k = 0xffff). A layer whose rows need
// more than kZMaxSlots slots keeps only the BF16 form (zcr = -1).
int encode_z(const LayerInfo &li, const void *W, LayerState &ns)
{
    const size_t n = (size_t)li.N * li.K;
    std::vector<uint16_t> h(n);
    hipError_t e = hipMemcpy(h.data(), W, n * 2, hipMemcpyDeviceToHost);
    if (e != hipSuccess)
        return hip_fail(e);
    size_t hist[128] = {0};
    for (size_t i = 0; i < n; ++i)
        ++hist[(h[i] >> 8) & 0x7f];
    int base = 0;
    size_t best = 0;
    for (int b = 0; b + 8 <= 128; ++b) {
        size_t c = 0;
        for (int j = 0; j < 8; ++j)
            c += hist[b + j];
        if (c > best) {
            best = c;
            base = b;
        }
    }
    std::vector<std::vector<uint64_t>> rows(li.N);
    size_t cr = 0;
    for (int r = 0; r < li.N; ++r) {
        for (int k = 0; k < li.K; ++k) {
            const uint32_t w = h[(size_t)r * li.K + k];
            const int hx = (int)((w >> 8) & 0x7fu);
            if (hx >= base && hx < base + 8)
                continue;
            const uint32_t c = (uint32_t)std::min(std::max(hx - base, 0), 7);
            const uint32_t d = (w & 0x8000u) | ((uint32_t)(base + (int)c) << 8) | (w & 0xffu);
            rows[r].push_back((uint64_t)k | ((uint64_t)w << 16) | ((uint64_t)d << 32));
        }
        cr = std::max(cr, rows[r].size());
        if (cr > (size_t)kZMaxSlots)
            return PROJ_OK;                   // too many corrections: BF16 form only
    }
    std::vector<uint64_t> tab((size_t)li.N * std::max<size_t>(cr, 1), 0xffffull);
    for (int r = 0; r < li.N; ++r)
        for (size_t j = 0; j < rows[r].size(); ++j)
            tab[(size_t)r * cr + j] = rows[r][j];
    if ((e = hipMalloc(reinterpret_cast<void **>(&ns.wz), n * 3 / 2)) != hipSuccess ||
        (e = hipMalloc(reinterpret_cast<void **>(&ns.zexc), tab.size() * 8)) != hipSuccess ||
        (e = hipMemcpy(ns.zexc, tab.data(), tab.size() * 8, hipMemcpyHostToDevice)) != hipSuccess)
        return hip_fail(e);
    hipLaunchKernelGGL(repack_z_kernel, dim3(4096), dim3(256), 0, nullptr, static_cast<const uint16_t *>(W), ns.wz,
                       li.N, li.K, base);
    if ((e = hipGetLastError()) != hipSuccess)
        return hip_fail(e);
    ns.zcr = (int)cr;
    ns.zt0 = (uint32_t)base | (uint32_t)(base + 1) << 8 | (uint32_t)(base + 2) << 16 | (uint32_t)(base + 3) << 24;
    ns.zt1 = (uint32_t)(base + 4) | (uint32_t)(base + 5) << 8 | (uint32_t)(base + 6) << 16 | (uint32_t)(base + 7) << 24;
    return PROJ_OK;
}

void free_layer(LayerState &st)
{
    if (st.wp)
        (void)hipFree(st.wp);
    if (st.ws)
        (void)hipFree(st.ws);
    if (st.counters)
        (void)hipFree(st.counters);
    if (st.pws)
        (void)hipFree(st.pws);
    if (st.zrow)
        (void)hipFree(st.zrow);
    if (st.wrow)
        (void)hipFree(st.wrow);
    if (st.wz)
        (void)hipFree(st.wz);
    if (st.zexc)
        (void)hipFree(st.zexc);
    if (st.giveups)
        (void)hipFree(st.giveups);
    st = LayerState{};
}

// Once per device, with that device current: the device address of the
// fixed scratch array, its polled region filled with the empty marks and the
// counters zeroed (the only writes to it outside the kernels themselves).
int scratch_setup(int dev)
{
    if (dev < 0 || dev >= kMaxDevices)
        return PROJ_ERR_DEVICE;
    if (g_scratch[dev])
        return PROJ_OK;
    void *p = nullptr;
    hipError_t e = hipGetSymbolAddress(&p, HIP_SYMBOL(scratch));
    if (e != hipSuccess)
        return hip_fail(e);
    if (!p)
        return PROJ_ERR_NULL;
    if ((e = hipMemset(p, 0xff, kScratchPolled)) != hipSuccess ||
        (e = hipMemset(static_cast<char *>(p) + kScratchPolled + kScratchCounted, 0,
                       kScratchCounters * sizeof(uint32_t))) != hipSuccess ||
        (e = hipDeviceSynchronize()) != hipSuccess)
        return hip_fail(e);
    g_scratch[dev] = p;
    return PROJ_OK;
}

// The layer state with its split-K workspaces replaced by the device's fixed
// scratch (capacities reduced to the scratch's regions).
LayerState with_scratch(const LayerState &st, void *p)
{
    LayerState v = st;
    char *b = static_cast<char *>(p);
    v.pws = reinterpret_cast<uint64_t *>(b);
    v.pws_bytes = kScratchPolled;
    v.ws = reinterpret_cast<f32x4 *>(b + kScratchPolled);
    v.ws_bytes = kScratchCounted;
    v.counters = reinterpret_cast<uint32_t *>(b + kScratchPolled + kScratchCounted);
    v.n_counters = kScratchCounters;
    return v;
}

// Launches every kernel the dispatch table can pick for the layer once (guide
// ch. 10 "Measure, experiment, and try your own changes", Experiment D: an
// unsupported configuration shows up in prepare's warm-up, never in a timed
// call). Every token count up to kPlanScanM is planned and resolved, so a
// table entry that is not compiled, or that does not tile the layer, fails
// prepare; each distinct kernel then runs once on zero activations, so its
// code object and first-launch cost are paid here and not inside a caller's
// graph capture or timed region.
int warm_up(int layer, const LayerState &ns)
{
    const LayerInfo &li = kLayers[layer];
    constexpr int kWarmM = kSliceMaxM + 1;          // past the unpooler slice
    void *zx = nullptr, *out = nullptr;
    hipError_t e;
    if ((e = hipMalloc(&zx, (size_t)kWarmM * li.K * 2)) != hipSuccess ||
        (e = hipMemset(zx, 0, (size_t)kWarmM * li.K * 2)) != hipSuccess ||
        (e = hipMalloc(&out, (size_t)kWarmM * li.N * li.o_bytes)) != hipSuccess) {
        (void)hipFree(zx);
        return hip_fail(e);
    }
    std::vector<const void *> done;
    int rc = PROJ_OK;
    for (int m = 1; m <= kPlanScanM && rc == PROJ_OK; ++m) {
        const proj_config c = plan_default(layer, m, ns.zcr);
        Launch L;
        if ((rc = resolve(layer, m, c, L, ns)) != PROJ_OK)
            break;
        if (std::find(done.begin(), done.end(), L.fn) != done.end())
            continue;
        done.push_back(L.fn);
        // The same configuration over one token (rows of the slice) or, for
        // the unpooler past its slice, over kWarmM tokens.
        const int mw = (layer == PROJ_UNPOOLER && m > kSliceMaxM) ? kWarmM : 1;
        Launch W;
        if ((rc = resolve(layer, mw, c, W, ns)) != PROJ_OK)
            break;
        rc = launch(W, zx, out, nullptr);
    }
    if (rc == PROJ_OK && (e = hipDeviceSynchronize()) != hipSuccess)
        rc = hip_fail(e);
    (void)hipFree(zx);
    (void)hipFree(out);
    return rc;
}

}  // namespace
}  // namespace gdp

using namespace gdp;

extern "C" {

int proj_prepare(int layer, const void *W)
{
    if (check_layer(layer))
        return PROJ_ERR_LAYER;
    if (!W)
        return PROJ_ERR_NULL;
    if (!aligned16(W))
        return PROJ_ERR_ALIGN;
    const LayerInfo &li = kLayers[layer];
    int dev = -1;
    hipError_t e = hipGetDevice(&dev);
    if (e != hipSuccess)
        return hip_fail(e);
    int rs = scratch_setup(dev);
    if (rs)
        return rs;
    // The new state is built, repacked and warmed up next to the old one,
    // which stays usable until the new one is complete.
    const size_t wbytes = (size_t)li.N * li.K * li.w_bytes;
    LayerState ns;
    ns.device = dev;
    if ((e = hipMalloc(&ns.wp, wbytes)) != hipSuccess ||
        (e = hipMalloc(reinterpret_cast<void **>(&ns.ws), kWsBytes)) != hipSuccess ||
        (e = hipMalloc(reinterpret_cast<void **>(&ns.counters), kCounters * sizeof(uint32_t))) != hipSuccess ||
        (e = hipMemset(ns.counters, 0, kCounters * sizeof(uint32_t))) != hipSuccess ||
        (e = hipMalloc(reinterpret_cast<void **>(&ns.pws), kWsBytes)) != hipSuccess ||
        (e = hipMemset(ns.pws, 0xff, kWsBytes)) != hipSuccess ||
        (e = hipMalloc(reinterpret_cast<void **>(&ns.giveups), 64)) != hipSuccess ||
        (e = hipMemset(ns.giveups, 0, 64)) != hipSuccess ||
        (e = hipMalloc(reinterpret_cast<void **>(&ns.zrow), (size_t)li.K * 2)) != hipSuccess ||
        (e = hipMemset(ns.zrow, 0, (size_t)li.K * 2)) != hipSuccess) {
        free_layer(ns);
        return hip_fail(e);
    }
    if (kRowMajorRows[layer] > 0) {
        const size_t rbytes = (size_t)kRowMajorRows[layer] * li.K * li.w_bytes;
        if ((e = hipMalloc(&ns.wrow, rbytes)) != hipSuccess ||
            (e = hipMemcpy(ns.wrow, W, rbytes, hipMemcpyDeviceToDevice)) != hipSuccess) {
            free_layer(ns);
            return hip_fail(e);
        }
        ns.wrow_rows = kRowMajorRows[layer];
    }
    const int threads = 256;
    const int blocks = 4096;
    if (li.w_bytes == 2) {
        hipLaunchKernelGGL(repack_bf16_kernel, dim3(blocks), dim3(threads), 0, nullptr,
                           static_cast<const uint16_t *>(W), static_cast<u32x4 *>(ns.wp), li.N, li.K);
        const int rc = encode_z(li, W, ns);
        if (rc) {
            free_layer(ns);
            return rc;
        }
    }
    else
        hipLaunchKernelGGL(repack_f32_kernel, dim3(blocks), dim3(threads), 0, nullptr,
                           static_cast<const float *>(W), static_cast<u32x4 *>(ns.wp), li.N, li.K);
    if ((e = hipGetLastError()) != hipSuccess || (e = hipDeviceSynchronize()) != hipSuccess) {
        free_layer(ns);
        return hip_fail(e);
    }
    const int rc = warm_up(layer, ns);
    if (rc) {
        free_layer(ns);
        return rc;
    }
    ns.prepared = true;
    free_layer(g_layers[layer]);
    g_layers[layer] = ns;
    return PROJ_OK;
}

int proj_run(int layer, const void *x, int m, void *out, void *stream)
{
    int rc = check_run_args(layer, x, m, out);
    if (rc)
        return rc;
    proj_config c = plan_default(layer, m, g_layers[layer].zcr);
    Launch L;
    rc = resolve(layer, m, c, L, g_layers[layer]);
    if (rc)
        return rc;
    return launch(L, x, out, static_cast<hipStream_t>(stream));
}

int proj_run_noalloc(int layer, const void *x, int m, void *out, void *stream)
{
    int rc = check_run_args(layer, x, m, out);
    if (rc)
        return rc;
    const LayerState &st = g_layers[layer];
    void *p = (st.device >= 0 && st.device < kMaxDevices) ? g_scratch[st.device] : nullptr;
    if (!p)
        return PROJ_ERR_NOT_PREPARED;
    proj_config c = plan_default(layer, m, st.zcr);
    Launch L;
    if ((rc = resolve(layer, m, c, L, st)) != PROJ_OK)
        return rc;
    // The same plan over the fixed scratch: only its capacity can refuse it.
    if (resolve(layer, m, c, L, with_scratch(st, p)) != PROJ_OK)
        return PROJ_ERR_SCRATCH;
    return launch(L, x, out, static_cast<hipStream_t>(stream));
}

int proj_run_config(int layer, const void *x, int m, void *out, void *stream, const proj_config *cfg)
{
    int rc = check_run_args(layer, x, m, out);
    if (rc)
        return rc;
    if (!cfg)
        return PROJ_ERR_NULL;
    Launch L;
    rc = resolve(layer, m, *cfg, L, g_layers[layer]);
    if (rc)
        return rc;
    return launch(L, x, out, static_cast<hipStream_t>(stream));
}

int proj_run_timed(int layer, const void *x, int m, void *out, void *stream, const proj_config *cfg,
                   void *ev_start, void *ev_stop)
{
    int rc = check_run_args(layer, x, m, out);
    if (rc)
        return rc;
    proj_config c = cfg ? *cfg : plan_default(layer, m, g_layers[layer].zcr);
    Launch L;
    rc = resolve(layer, m, c, L, g_layers[layer]);
    if (rc)
        return rc;
    return launch(L, x, out, static_cast<hipStream_t>(stream), static_cast<hipEvent_t>(ev_start),
                  static_cast<hipEvent_t>(ev_stop));
}

int proj_plan(int layer, int m, proj_config *cfg)
{
    if (check_layer(layer))
        return PROJ_ERR_LAYER;
    if (m < 1 || m > kMaxM)
        return PROJ_ERR_M;
    if (!cfg)
        return PROJ_ERR_NULL;
    proj_config c = plan_default(layer, m, g_layers[layer].zcr);
    Launch L;
    int rc = resolve(layer, m, c, L, g_layers[layer]);
    if (rc)
        return rc;
    c.grid = L.grid;
    c.block = L.block;
    *cfg = c;
    return PROJ_OK;
}

int proj_out_cols(int layer, int m)
{
    if (check_layer(layer))
        return PROJ_ERR_LAYER;
    if (m < 1 || m > kMaxM)
        return PROJ_ERR_M;
    return n_eff_of(layer, m);
}

int proj_layer_dims(int layer, int *N, int *K, int *w_elem_bytes, int *out_elem_bytes)
{
    if (check_layer(layer))
        return PROJ_ERR_LAYER;
    const LayerInfo &li = kLayers[layer];
    if (N) *N = li.N;
    if (K) *K = li.K;
    if (w_elem_bytes) *w_elem_bytes = li.w_bytes;
    if (out_elem_bytes) *out_elem_bytes = li.o_bytes;
    return PROJ_OK;
}

int proj_release(int layer)
{
    if (check_layer(layer))
        return PROJ_ERR_LAYER;
    free_layer(g_layers[layer]);
    return PROJ_OK;
}

const char *proj_strerror(int status)
{
    switch (status) {
    case PROJ_OK: return "ok";
    case PROJ_ERR_LAYER: return "unknown layer id";
    case PROJ_ERR_M: return "token count m out of range";
    case PROJ_ERR_NULL: return "null pointer";
    case PROJ_ERR_ALIGN: return "pointer not 16-byte aligned";
    case PROJ_ERR_NOT_PREPARED: return "layer not prepared";
    case PROJ_ERR_UNSUPPORTED: return "kernel configuration not compiled or does not tile the layer";
    case PROJ_ERR_HIP: return "HIP runtime error";
    case PROJ_ERR_DEVICE: return "current device differs from the layer's or the tensors'";
    case PROJ_ERR_SCRATCH: return "the plan's split-K partials exceed the fixed scratch of proj_run_noalloc";
    case PROJ_ERR_ARG: return "a size, stride, type or index is outside what the operator takes";
    case PROJ_ERR_PAGES: return "too few free pages in the pool";
    default: return "unknown status";
    }
}

int proj_last_hip_error(void) { return g_last_hip; }

int proj_num_variants(void) { return total_variants(); }

int proj_variant(int i, int *is_f32w, proj_config *cfg)
{
    const int wide0 = skinny_variants() + kTiledVariantCount + kRowVariantCount;
    if (i >= wide0 && i < total_variants()) {
        const WideVariant &w = wide_variant_at(i - wide0);
        if (is_f32w)
            *is_f32w = w.f32w;
        if (cfg) {
            proj_config c{};
            c.kind = 3;
            c.nt = w.bnb;
            c.rb = w.bmb;
            c.waves = w.waves;
            c.spw = w.depth;
            c.ksplit = 1;
            c.block = w.waves * kWave;
            c.flags = w.xdma ? kFlagDma : 0;
            *cfg = c;
        }
        return PROJ_OK;
    }
    if (i >= skinny_variants() + kTiledVariantCount && i < wide0) {
        const RowVariant &r = kRowVariants[i - skinny_variants() - kTiledVariantCount];
        if (is_f32w)
            *is_f32w = r.f32w;
        if (cfg) {
            proj_config c{};
            c.kind = 2;
            c.nt = r.mcap;
            c.rb = r.r;
            c.waves = kRowWaves;
            c.spw = r.kit;
            c.ksplit = 1;
            c.block = kRowThreads;
            *cfg = c;
        }
        return PROJ_OK;
    }
    if (i >= skinny_variants() && i < total_variants()) {
        const TiledVariant &t = kTiledVariants[i - skinny_variants()];
        if (is_f32w)
            *is_f32w = t.f32w;
        if (cfg) {
            proj_config c{};
            c.kind = 1;
            c.nt = t.bnb;
            c.rb = t.bmb;
            c.waves = t.wr * t.kg;
            c.spw = t.depth;
            c.ksplit = 1;
            c.block = c.waves * kWave;
            *cfg = c;
        }
        return PROJ_OK;
    }
    const SkinnyVariant *v = variant_at(i);
    if (!v)
        return PROJ_ERR_UNSUPPORTED;
    if (is_f32w)
        *is_f32w = v->f32w;
    if (cfg) {
        proj_config c{};
        c.kind = 0;
        c.nt = v->nt;
        c.rb = v->rb;
        c.waves = v->waves;
        c.spw = v->spw;
        c.ksplit = 1;
        c.flags = (v->z ? 4 : 0) | (v->xp == 4 ? kFlagPreload4 : v->xp == 8 ? kFlagPreload8 : 0) |
                  (v->skm ? kFlagStream : 0);
        c.block = (v->waves + v->z) * kWave;
        *cfg = c;
    }
    return PROJ_OK;
}

int proj_split_giveups(int layer, int reset)
{
    if (check_layer(layer))
        return PROJ_ERR_LAYER;
    const LayerState &st = g_layers[layer];
    if (!st.prepared)
        return PROJ_ERR_NOT_PREPARED;
    int dev = -1;
    hipError_t e = hipGetDevice(&dev);
    if (e != hipSuccess)
        return hip_fail(e);
    if (dev != st.device)
        return PROJ_ERR_DEVICE;
    uint32_t n = 0;
    if ((e = hipDeviceSynchronize()) != hipSuccess ||
        (e = hipMemcpy(&n, st.giveups, sizeof n, hipMemcpyDeviceToHost)) != hipSuccess)
        return hip_fail(e);
    if (reset) {
        // A partial published after its reducer gave up would read as
        // arrived in a later launch: restore every mark (the layer's
        // workspace and the device's fixed scratch), then the count.
        void *p = (st.device >= 0 && st.device < kMaxDevices) ? g_scratch[st.device] : nullptr;
        if ((p && (e = hipMemset(p, 0xff, kScratchPolled)) != hipSuccess) ||
            (e = hipMemset(st.pws, 0xff, kWsBytes)) != hipSuccess ||
            (e = hipMemset(st.giveups, 0, sizeof n)) != hipSuccess || (e = hipDeviceSynchronize()) != hipSuccess)
            return hip_fail(e);
    }
    return (int)(n > 0x7fffffffu ? 0x7fffffffu : n);
}

int proj_compressed(int layer)
{
    if (check_layer(layer))
        return PROJ_ERR_LAYER;
    const LayerState &st = g_layers[layer];
    if (!st.prepared)
        return PROJ_ERR_NOT_PREPARED;
    return st.zcr < 0 ? -1 : st.zcr;
}

}  // extern "C"
