// C ABI of an 8-bit base model's operators (include/lora_w8.h): argument checks and launch.
#include <string.h>

#include <algorithm>

#include "host.h"
#include "q8_rows.cuh"
#include "w8_narrow.cuh"
#include "w8_wide.cuh"

using namespace lora;
using namespace lora::host;

namespace {

// ---------------------------------------------------------------------------- rows in 8 bits
// A 16-bit matrix of rows of width d.
lora_status check_rows(const void* p, int64_t ld, int32_t d) {
    if (p == nullptr) return LORA_EINVAL;
    if (!aligned16(p) || ld % 8 != 0) return LORA_EALIGN;
    return ld >= d ? LORA_OK : LORA_EINVAL;
}

lora_status check_out(const lora_q8_rows& o, int32_t d) {
    if (o.codes == nullptr || o.scales == nullptr || o.reserved != 0) return LORA_EINVAL;
    if (o.x_kind != LORA_Q8_X_HELD && o.x_kind != LORA_Q8_X_FULL) return LORA_EINVAL;
    if (!aligned16(o.codes) || o.ldc % 16 != 0 || ((uintptr_t)o.scales & 3u) != 0) return LORA_EALIGN;
    if (o.ldc < d) return LORA_EINVAL;
    return o.x != nullptr ? check_rows(o.x, o.ldx, d) : LORA_OK;
}

lora_status check_shape(int32_t T, int32_t d) {
    if (T < 0 || d <= 0 || d % 16 != 0) return LORA_EINVAL;
    return T > LORA_Q8_MAX_ROWS || d > LORA_Q8_MAX_WIDTH ? LORA_ETOOBIG : LORA_OK;
}

// In place is fine where both sides have one pitch.
bool pitch_differs(const void* a, int64_t lda, const void* b, int64_t ldb) { return a != nullptr && a == b && lda != ldb; }

Q8Out out_of(const lora_q8_rows& o) {
    return {reinterpret_cast<unsigned char*>(o.codes), o.scales, reinterpret_cast<__nv_bfloat16*>(o.x), o.ldc, o.ldx,
            o.x_kind == LORA_Q8_X_FULL};
}

// A launch that is made ready while the kernel before it in the stream still runs; the kernel waits for that one's end by
// grid_wait().  In a graph, us: one row of 4096 x 4096 (in L2) 4.2 -> 3.9, 8,191 rows of the norm 49.5 -> 49.0; called one behind
// the other 13 rows of q, k, v (in L2) 10.4 -> 7.4, 2,339 gated rows 41.4 -> 38.9, 64 rows of 117 MB 29.5 -> 27.5.  Where the few-row
// kernel lets the next one begin while it runs, that one's CTAs take uneven places: 3.9 -> 5.0, 7.1 -> 7.9.
template <typename P>
lora_status launch_early(void (*kern)(P), dim3 grid, int threads, size_t smem, cudaStream_t s, const P& p) {
    cudaLaunchAttribute early;
    early.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    early.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.attrs = &early;
    cfg.numAttrs = 1;
    cfg.stream = s;
    return cuda_status(cudaLaunchKernelEx(&cfg, kern, p));
}

// Threads of a row, and CTAs: every row its own while the SMs hold them all, else as many as the
// SMs hold (1,024 threads, at the kernels' 64 registers), each with rows in turn.
template <typename K, typename P>
lora_status launch_rows(K kern, const P& q, int v, cudaStream_t s) {
    DeviceInfo* di = nullptr;
    lora_status st = device_info(&di);
    if (st != LORA_OK) return st;
    const int threads = ((q.d / 8 + v - 1) / v + 31) / 32 * 32;
    return launch_early(kern, dim3(std::min(q.T, di->sm_count * std::max(1024 / threads, 1))), threads, 0, s, q);
}

// Eights of a row that a thread holds, by measured times: a norm's weights fit beside one of them and
// the next row (8,191 rows of 4096: 49 us, 59 with two), above that several CTAs an SM with four each
// and nothing ahead are better (8,000 of 5120: 70 with one, 76 with two, 64, 86% of a copy's rate; 2,000 of 14336:
// 67 with two, 50 to 54, 72 to 78%).  An activation has no weights: two and the next row (2,339 gated of 14336 39, 50 with
// four; 8,000 of 4096 without a gate 29, 36 with one), for narrow rows one.
template <int ACT>
lora_status launch_gate(const Q8GateParams& q, cudaStream_t s) {
    if (q.d <= 2048) return launch_rows(q8_gate_kernel<1, ACT, true>, q, 1, s);
    if (q.d <= 16384) return launch_rows(q8_gate_kernel<2, ACT, true>, q, 2, s);
    return launch_rows(q8_gate_kernel<4, ACT, false>, q, 4, s);
}
lora_status launch_norm(const Q8NormParams& q, cudaStream_t s) {
    if (q.d <= 4096) return launch_rows(q8_norm_kernel<1, true>, q, 1, s);
    return launch_rows(q8_norm_kernel<4, false>, q, 4, s);
}

// ---------------------------------------------------------------------------- products
lora_status check_sizes(const lora_w8_problem* probs, int32_t nprob, int32_t T) {
    if (nprob < 0 || T < 0 || (nprob > 0 && probs == nullptr)) return LORA_EINVAL;
    if (nprob > LORA_W8_MAX_PROBLEMS || T > LORA_W8_MAX_ROWS) return LORA_ETOOBIG;
    for (int32_t i = 0; i < nprob; ++i) {
        const lora_w8_problem& p = probs[i];
        if (p.N <= 0 || p.K <= 0 || p.N % 8 != 0 || p.K % 16 != 0) return LORA_EINVAL;
        if (p.N > (1 << 24) || p.K > LORA_W8_MAX_K) return LORA_ETOOBIG;
    }
    return LORA_OK;
}

// Which kernel serves.  w8_narrow.cuh begins 5 us earlier than w8_wide.cuh, but takes W through the SMs once
// per 32 rows of x and widens x once per 16 rows of W.  Narrow and wide, us, W from memory: 16 rows of 17 MB
// 6.8 and 14.4, 25 MB 10.5 and 16.1, 50 MB 16.1 and 16.5, 59 MB in rows of 14336 16.7 and 21.5, 79 MB 22.8 and 19.9,
// 117 MB 31 and 27.  From 17 rows on an SM holds one narrow CTA, whose time goes by K; the wide kernel joins its
// sums where K is long: 32 rows of 4 MB 5.9 and 13.0, 17 MB 10.9 and 14.2, 25 MB 15.6 and 16.2, 50 MB 28.7 and
// 16.6, 59 MB in rows of 14336 26.4 and 21.7, 17 MB in rows of 1024 19.2 and 9.7; 64 rows of 8 MB 9.9 and 14.4,
// 17 MB 18.2 and 16.0; 128 rows of 4 MB 10.0 and 14.4, 8 MB 17.2 and 15.5; 300 rows of 4 MB 21.0 and 15.7.  The
// estimate, fitted with W in L2, takes the faster one at each of these.  152 SMs: a workspace's size is asked for
// without a device.  A call that is narrow is so for fewer rows too: a workspace serves those.
constexpr int64_t kW8Narrow16 = 58 << 20;
bool narrow(const lora_w8_problem* probs, int32_t nprob, int32_t T) {
    if (T <= 8) return true;
    int64_t bytes = 0, tiles = 0, k = 0;
    for (int32_t i = 0; i < nprob; ++i) {
        bytes += (int64_t)probs[i].N * probs[i].K;
        tiles += (probs[i].N + kW8Rows - 1) / kW8Rows;
        k = std::max<int64_t>(k, probs[i].K);
    }
    if (bytes > kW8Narrow16) return false;
    if (T <= 16) return true;
    const int64_t turns = (tiles * ((T + 31) / 32) + 151) / 152;                      // CTAs of an SM, one by one
    const int64_t narrow_ns = 2000 + turns * (1100 + k * 58 / 100);
    const int64_t wide_ns = 4300 + std::min<int64_t>(7600, k * 34 / 10) + bytes / 10000;
    return narrow_ns <= wide_ns;
}

// How a wide call is shared out.
struct WideShape {
    int cols, ttiles;              // columns of a tile (rows of x), tiles along x
    int32_t per;                   // steps of a pair
    bool split;                    // whether a pair's range begins or ends inside a tile
};
constexpr int wide_max(int cols) { return cols <= 64 ? 64 : cols <= 128 ? 128 : 256; }

// The number of tiles along x, whole or in equal shares of all steps, that should take the fewest clocks: a
// step of c columns takes 4 c for its MMAs, 620 for its widening, and 870 for its W from memory where
// all pairs stream and no other tile has fetched it; a tile of more than 128 columns, whose sums leave before
// the next one's begin, 5,000 at its end; joining a tile from several pairs 6,000 + 100 c, and
// 18 c for each part past the second.  us: 700 rows of 4096 x 14336 63 in shares of tiles of 256, 56 in whole ones of 192, 58 in shares
// of 160; 300 rows 36 in shares of 160, 46 whole, 41 in whole ones of 128; 500 rows of it 50 in
// shares of 256, 43 in whole ones of 128; 200 rows of three 5120 x 5120 29 in whole tiles of 224, 35 in
// shares of them, 34 in whole ones of 128; 600 rows of two 14336 x 4096 90 in shares of 224, 86 in whole ones
// of 160.  A share is not so small that a tile has many parts (35 rows of 184 x 6400: 28 us in 50 parts,
// 13 in 9; 100 rows of 4096 x 4096 19 in 6, 15 in 4).
WideShape wide_shape(const lora_w8_problem* probs, int32_t nprob, int32_t T, int pairs) {
    WideShape best = {0, 0, 0, false};
    int64_t least = INT64_MAX, rows = 0, blocks = 0;               // tiles along W, and their steps
    int32_t kb = 0;
    bool one_k = true;
    for (int32_t i = 0; i < nprob; ++i) {
        const int32_t k = (probs[i].K + kW8WideK - 1) / kW8WideK;
        const int64_t n = (probs[i].N + kW8WideRows - 1) / kW8WideRows;
        one_k = one_k && (i == 0 || k == kb);
        kb = std::max(kb, k);
        rows += n;
        blocks += n * k;
    }
    const int fewest = (T + 255) / 256, most = (T + 63) / 64;
    for (const int about : {fewest, fewest + 1, fewest + 2, fewest + 3, (T + 127) / 128, most}) {
        if (about > most) continue;
        const int cols = ((T + about - 1) / about + 31) / 32 * 32, ttiles = (T + cols - 1) / cols;
        const int64_t tiles = rows * ttiles, steps = blocks * ttiles, drain = cols > 128 ? 5000 : 0;
        auto clocks = [&](int64_t per) {
            const int64_t busy = std::min<int64_t>(pairs, (steps + per - 1) / per);
            return per * std::max<int64_t>({620, 4 * cols, 870 * busy / pairs / ttiles});
        };
        const int64_t share = std::max<int64_t>((steps + pairs - 1) / pairs, cols <= 64 ? 6 : 10);
        const int64_t in_shares = clocks(share) + 6000 + 100 * cols + std::max<int64_t>(share / kb - 1, 0) * drain +
                                  std::max<int64_t>(kb - 2 * share, 0) * 18 * cols / share;
        if (in_shares < least) {
            least = in_shares;
            best = {cols, ttiles, (int32_t)std::min<int64_t>(share, INT32_MAX), true};
        }
        const int64_t whole = (tiles + pairs - 1) / pairs * kb;
        const int64_t as_whole = clocks(whole) + std::max<int64_t>(whole / kb * drain, 2000);
        if (one_k && as_whole < least) {
            least = as_whole;
            best = {cols, ttiles, (int32_t)std::min<int64_t>(whole, INT32_MAX), false};
        }
    }
    return best;
}

// The first problem with i's x.
int32_t x_of(const lora_w8_problem* probs, int32_t i) {
    int32_t j = 0;
    while (probs[j].x != probs[i].x || probs[j].ldx != probs[i].ldx || probs[j].K != probs[i].K) ++j;
    return j;
}

size_t x_bytes(const lora_w8_problem& p, int32_t T) { return align256((size_t)T * p.K * 2); }

size_t workspace_bytes(const lora_w8_problem* probs, int32_t nprob, int32_t T) {
    if (narrow(probs, nprob, T)) return align256(kStepPartAt);
    size_t n = align256(kStepPartAt) + w8_part_bytes(wide_max(std::min(T, 256)));   // of the widest tiles
    for (int32_t i = 0; i < nprob; ++i)
        if (x_of(probs, i) == i) n += x_bytes(probs[i], T);
    return n;
}

template <int MAX>
lora_status run_narrow(const lora_w8_problem* probs, int32_t nprob, int32_t T, cudaStream_t s) {
    W8Params<MAX> p;
    p.T = T;
    p.nprob = nprob;
    int64_t total = 0;
    uint64_t at = 0;
    for (int32_t i = 0; i < nprob; ++i) {
        const lora_w8_problem& pr = probs[i];
        at |= (uintptr_t)pr.x | (uintptr_t)pr.w | (uint64_t)pr.ldx | (uint64_t)pr.K;
        p.prob[i] = {reinterpret_cast<const unsigned char*>(pr.x), pr.x_scales, reinterpret_cast<__nv_bfloat16*>(pr.y),
                     reinterpret_cast<const unsigned char*>(pr.w), pr.w_scales, pr.ldx, pr.ldy, pr.N, pr.K, (int32_t)total};
        total += (pr.N + kW8Rows - 1) / kW8Rows;
    }
    p.total = (int32_t)total;
    const int nt = T <= 8 ? 1 : T <= 16 ? 2 : 4;
    const dim3 grid((unsigned)total, (unsigned)((T + 31) / 32));
    const bool by32 = at % 32 == 0;
    void (*kern)(W8Params<MAX>) = nt == 1 ? (by32 ? w8_narrow_kernel<1, MAX, true> : w8_narrow_kernel<1, MAX, false>)
                                : nt == 2 ? (by32 ? w8_narrow_kernel<2, MAX, true> : w8_narrow_kernel<2, MAX, false>)
                                          : (by32 ? w8_narrow_kernel<4, MAX, true> : w8_narrow_kernel<4, MAX, false>);
    return launch_early(kern, grid, kW8Threads, 0, s, p);
}

// 2-D map of `rows` rows of `inner` elements, box {box0, box1}, zeros outside.
lora_status map2d(PFN_cuTensorMapEncodeTiled_v12000 enc, CUtensorMap* map, CUtensorMapDataType type, const void* base,
                  uint64_t inner, uint64_t rows, uint64_t pitch, uint32_t box0, uint32_t box1, CUtensorMapSwizzle swizzle) {
    const cuuint64_t dims[2] = {inner, rows};
    const cuuint64_t strides[1] = {pitch};
    const cuuint32_t box[2] = {box0, box1}, one[2] = {1, 1};
    const CUresult r = enc(map, type, 2, const_cast<void*>(base), dims, strides, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE,
                           swizzle, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    if (r == CUDA_SUCCESS) return LORA_OK;
    g_last_cuda_error = 10000 + (int)r;
    return LORA_ECUDA;
}

// Readies a kernel on the current device, once; pairs of CTAs that the device holds at a time.
template <int NMAX, bool SPLIT>
lora_status ready_wide(int* out) {
    DeviceInfo* di = nullptr;
    lora_status st = device_info(&di);
    if (st != LORA_OK) return st;
    auto kern = w8_wide_kernel<NMAX, SPLIT>;
    static thread_local const DeviceInfo* ready = nullptr;
    static thread_local int pairs = 0;
    if (ready != di) {
        cudaLaunchAttribute pair;
        pair.id = cudaLaunchAttributeClusterDimension;
        pair.val.clusterDim.x = 2;
        pair.val.clusterDim.y = pair.val.clusterDim.z = 1;
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3(di->sm_count / 2 * 2);
        cfg.blockDim = dim3(kW8WideThreads);
        cfg.dynamicSmemBytes = w8_wide_smem(NMAX);
        cfg.attrs = &pair;
        cfg.numAttrs = 1;
        st = cuda_status(cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)cfg.dynamicSmemBytes));
        if (st != LORA_OK) return st;
        st = cuda_status(cudaOccupancyMaxActiveClusters(&pairs, kern, &cfg));
        if (st != LORA_OK) return st;
        pairs = std::max(1, std::min(pairs, kW8MaxPairs));
        ready = di;
    }
    *out = pairs;
    return LORA_OK;
}

template <int NMAX, bool SPLIT>
lora_status launch_wide(const W8WideParams& w, int pairs, cudaStream_t s) {
    return launch_early(w8_wide_kernel<NMAX, SPLIT>, dim3(2 * pairs), kW8WideThreads, w8_wide_smem(NMAX), s, w);
}

template <int NMAX>
lora_status launch_wide(const W8WideParams& w, bool split, int pairs, cudaStream_t s) {
    return split ? launch_wide<NMAX, true>(w, pairs, s) : launch_wide<NMAX, false>(w, pairs, s);
}

// Pairs of CTAs that the device holds, all kernels ready.
lora_status ready_wide(int* pairs) {
    lora_status st = LORA_OK;
    *pairs = kW8MaxPairs;
    int n = 0;
    auto take = [&](lora_status r) {
        if (st == LORA_OK) st = r;
        *pairs = std::min(*pairs, n);
    };
    take(ready_wide<64, false>(&n));
    take(ready_wide<64, true>(&n));
    take(ready_wide<128, false>(&n));
    take(ready_wide<128, true>(&n));
    take(ready_wide<256, false>(&n));
    take(ready_wide<256, true>(&n));
    return st;
}

lora_status run_wide(const lora_w8_problem* probs, int32_t nprob, int32_t T, void* ws, cudaStream_t s, int32_t lost,
                     uint64_t limit_ns) {
    PFN_cuTensorMapEncodeTiled_v12000 enc = nullptr;
    lora_status st = encode_fn(&enc);
    if (st != LORA_OK) return st;
    static thread_local W8WideParams w;
    static thread_local W8Widen v;
    memset(&w, 0, sizeof w);
    memset(&v, 0, sizeof v);
    int pairs = 0;
    if ((st = ready_wide(&pairs)) != LORA_OK) return st;
    const WideShape sh = wide_shape(probs, nprob, T, pairs);
    const int nmax = wide_max(sh.cols);
    char* base = reinterpret_cast<char*>(ws);
    w.nprob = nprob;
    w.T = v.T = T;
    w.cols = sh.cols;
    w.ttiles = sh.ttiles;
    w.tickets = reinterpret_cast<uint32_t*>(base + sizeof(WsHeader));
    w.part = reinterpret_cast<float*>(base + align256(kStepPartAt));
    w.err = &reinterpret_cast<WsHeader*>(ws)->err;
    w.limit_ns = limit_ns;
    w.lost = lost;
    char* at = base + align256(kStepPartAt) + w8_part_bytes(nmax);
    int32_t copies = 0, slot[LORA_W8_MAX_PROBLEMS];
    int64_t total = 0, most = 0;
    for (int32_t i = 0; i < nprob; ++i) {
        const lora_w8_problem& pr = probs[i];
        const int32_t j = x_of(probs, i);
        if (j == i) {
            v.x[copies] = reinterpret_cast<const unsigned char*>(pr.x);
            v.out[copies] = reinterpret_cast<uint32_t*>(at);
            v.ldx[copies] = pr.ldx;
            v.K[copies] = pr.K;
            most = std::max(most, (int64_t)T * (pr.K / 16));
            st = map2d(enc, &w.x[copies], CU_TENSOR_MAP_DATA_TYPE_FLOAT16, at, pr.K, T, (uint64_t)pr.K * 2, 64, sh.cols / 2,
                       CU_TENSOR_MAP_SWIZZLE_128B);
            if (st != LORA_OK) return st;
            at += x_bytes(pr, T);
            slot[i] = copies++;
        } else {
            slot[i] = slot[j];
        }
        st = map2d(enc, &w.w[i], CU_TENSOR_MAP_DATA_TYPE_UINT8, pr.w, pr.K, pr.N, pr.K, kW8WideK, 128, CU_TENSOR_MAP_SWIZZLE_128B);
        if (st != LORA_OK) return st;
        w.prob[i] = {pr.x_scales, pr.w_scales, reinterpret_cast<__nv_bfloat16*>(pr.y), pr.ldy, pr.N, (pr.K + kW8WideK - 1) / kW8WideK, (int32_t)total, slot[i]};
        total += (int64_t)((pr.N + kW8WideRows - 1) / kW8WideRows) * sh.ttiles * w.prob[i].kblocks;
        if (total > (1 << 30)) return LORA_ETOOBIG;
    }
    if (lost >= total) return LORA_EINVAL;
    w.total = (int32_t)total;
    pairs = std::min(pairs, (w.total + sh.per - 1) / sh.per);
    w.per = sh.per;
    if (!sh.split) {
        const int32_t kb = w.prob[0].kblocks, tiles = w.total / kb;
        w.per = tiles / pairs;
        w.more = tiles % pairs;
        w.over_rt = pairs / sh.ttiles;
        w.over_tt = pairs % sh.ttiles;
        if (lost >= 0) {
            w.lost_pair = lost / kb % pairs;
            w.lost = lost / kb / pairs * kb + lost % kb;
        }
    }
    DeviceInfo* di = nullptr;
    if ((st = device_info(&di)) != LORA_OK) return st;
    const int64_t blocks = std::min<int64_t>((most + kWidenThreads - 1) / kWidenThreads, std::max(di->sm_count * 8 / copies, 1));
    st = launch_early(w8_widen_kernel, dim3((unsigned)blocks, (unsigned)copies), kWidenThreads, 0, s, v);
    if (st != LORA_OK) return st;
    if (nmax == 64) return launch_wide<64>(w, sh.split, pairs, s);
    return nmax == 128 ? launch_wide<128>(w, sh.split, pairs, s) : launch_wide<256>(w, sh.split, pairs, s);
}

lora_status run(const lora_w8_problem* probs, int32_t nprob, int32_t T, void* ws, size_t ws_bytes, void* stream, int32_t lost,
                uint64_t limit_ns) {
    lora_status st = check_sizes(probs, nprob, T);
    if (st != LORA_OK) return st;
    for (int32_t i = 0; i < nprob; ++i) {
        const lora_w8_problem& pr = probs[i];
        if (pr.x == nullptr || pr.x_scales == nullptr || pr.y == nullptr || pr.w == nullptr || pr.w_scales == nullptr) return LORA_EINVAL;
        if (!aligned16(pr.x) || !aligned16(pr.y) || !aligned16(pr.w) || ((uintptr_t)pr.x_scales & 3u) != 0 ||
            ((uintptr_t)pr.w_scales & 3u) != 0 || pr.ldx % 16 != 0 || pr.ldy % 8 != 0)
            return LORA_EALIGN;
        if (pr.ldx < pr.K || pr.ldy < pr.N) return LORA_EINVAL;
    }
    if (nprob == 0 || T == 0) return LORA_OK;
    if (ws == nullptr || ((uintptr_t)ws & 255u) != 0 || ws_bytes < workspace_bytes(probs, nprob, T)) return LORA_EWORKSPACE;
    cudaStream_t s = (cudaStream_t)stream;
    if (!narrow(probs, nprob, T)) return run_wide(probs, nprob, T, ws, s, lost, limit_ns);
    return nprob <= 3 ? run_narrow<3>(probs, nprob, T, s) : run_narrow<LORA_W8_MAX_PROBLEMS>(probs, nprob, T, s);
}

}  // namespace

extern "C" {

lora_status lora_q8_norm(const lora_q8_norm_desc* n, int32_t T, void* stream) {
    if (n == nullptr) return LORA_EINVAL;
    lora_status st = check_shape(T, n->d);
    if (st != LORA_OK) return st;
    if (!(n->eps >= 1e-30f) || !(n->eps <= 1.f)) return LORA_EINVAL;
    if ((st = check_rows(n->x, n->ldx, n->d)) != LORA_OK) return st;
    if (n->residual != nullptr && (st = check_rows(n->residual, n->ldr, n->d)) != LORA_OK) return st;
    if (n->sum != nullptr && n->residual == nullptr) return LORA_EINVAL;
    if (n->sum != nullptr && (st = check_rows(n->sum, n->lds, n->d)) != LORA_OK) return st;
    if ((st = check_rows(n->weight, n->d, n->d)) != LORA_OK) return st;
    if (pitch_differs(n->sum, n->lds, n->x, n->ldx) || pitch_differs(n->sum, n->lds, n->residual, n->ldr)) return LORA_EINVAL;
    if ((st = check_out(n->out, n->d)) != LORA_OK) return st;
    if (T == 0) return LORA_OK;
    const Q8NormParams q = {reinterpret_cast<const __nv_bfloat16*>(n->x), reinterpret_cast<const __nv_bfloat16*>(n->residual),
                            reinterpret_cast<__nv_bfloat16*>(n->sum), reinterpret_cast<const __nv_bfloat16*>(n->weight),
                            n->ldx, n->ldr, n->lds, n->eps, 1.f / (float)n->d, n->d, T, out_of(n->out)};
    return launch_norm(q, (cudaStream_t)stream);
}

lora_status lora_q8_gate(const lora_q8_gate_desc* n, int32_t T, void* stream) {
    if (n == nullptr) return LORA_EINVAL;
    lora_status st = check_shape(T, n->d);
    if (st != LORA_OK) return st;
    if (n->act < LORA_ACT_NONE || n->act > LORA_ACT_GELU_TANH) return LORA_EINVAL;
    if ((st = check_rows(n->gate, n->ldg, n->d)) != LORA_OK) return st;
    if (n->up != nullptr && (st = check_rows(n->up, n->ldu, n->d)) != LORA_OK) return st;
    if ((st = check_out(n->out, n->d)) != LORA_OK) return st;
    if (pitch_differs(n->out.x, n->out.ldx, n->gate, n->ldg) || pitch_differs(n->out.x, n->out.ldx, n->up, n->ldu)) return LORA_EINVAL;
    if (T == 0) return LORA_OK;
    const Q8GateParams q = {reinterpret_cast<const __nv_bfloat16*>(n->gate), reinterpret_cast<const __nv_bfloat16*>(n->up),
                            n->ldg, n->ldu, n->d, T, out_of(n->out)};
    cudaStream_t s = (cudaStream_t)stream;
    switch (n->act) {
        case LORA_ACT_NONE: return launch_gate<LORA_ACT_NONE>(q, s);
        case LORA_ACT_SILU: return launch_gate<LORA_ACT_SILU>(q, s);
        case LORA_ACT_GELU: return launch_gate<LORA_ACT_GELU>(q, s);
        default: return launch_gate<LORA_ACT_GELU_TANH>(q, s);
    }
}

lora_status lora_w8_workspace_size(const lora_w8_problem* probs, int32_t nprob, int32_t T, size_t* bytes) {
    if (bytes == nullptr) return LORA_EINVAL;
    lora_status st = check_sizes(probs, nprob, T);
    if (st != LORA_OK) return st;
    *bytes = workspace_bytes(probs, nprob, T);
    return LORA_OK;
}

lora_status lora_w8_matmul(const lora_w8_problem* probs, int32_t nprob, int32_t T, void* ws, size_t ws_bytes, void* stream) {
    return run(probs, nprob, T, ws, ws_bytes, stream, -1, kWaitLimitNs);
}

lora_status lora_debug_w8_lost_step(const lora_w8_problem* probs, int32_t nprob, int32_t T, int32_t step, uint64_t limit_ns,
                                    void* ws, size_t ws_bytes, void* stream) {
    lora_status st = check_sizes(probs, nprob, T);
    if (st != LORA_OK) return st;
    if (narrow(probs, nprob, T) || step < 0 || limit_ns < 1000000ull) return LORA_EINVAL;
    if (limit_ns > kWaitLimitNs) return LORA_ETOOBIG;
    return run(probs, nprob, T, ws, ws_bytes, stream, step, limit_ns);
}

}  // extern "C"
