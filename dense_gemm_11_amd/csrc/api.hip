// C ABI of the dense GEMM library: argument validation, degenerate cases,
// per-shape kernel selection and the launch.  Declared in include/dense_gemm.h.
#include <algorithm>
#include <atomic>
#include <climits>
#include <cstdio>
#include <cstdlib>
#include <cstring>
#include <mutex>
#include <new>
#include <vector>

#include "dense_gemm.h"
#include "common.hpp"
#include "handle.hpp"
#include "variants.hpp"
#include "sk_ranges.hpp"

namespace dg {

// D = beta * C (or 0 when beta == 0), then the fused epilogue (bias,
// activation, clamp; nothing for a plain call): the whole result when K == 0
// or alpha == 0.
template <typename OutT>
__global__ __launch_bounds__(256) void scale_c_kernel(GemmArgs p)
{
    const int64_t total = (int64_t)p.M * p.N;
    const OutT* C = reinterpret_cast<const OutT*>(p.C);
    OutT* D = reinterpret_cast<OutT*>(p.D);
    for (int64_t e = (int64_t)blockIdx.x * 256 + threadIdx.x; e < total;
         e += (int64_t)gridDim.x * 256) {
        const int64_t row = e / p.N, col = e % p.N;
        const float v = (p.beta != 0.0f) ? p.beta * to_f32(C[row * p.ldc + col]) : 0.0f;
        D[row * p.ldd + col] = from_f32<OutT>(epilogue_op(p, v, bias_of<OutT>(p, (int)col)));
    }
}


// Zero the stream-K flags of a workspace.
__global__ __launch_bounds__(256) void clear_flags_kernel(unsigned* flags, int n)
{
    for (int i = blockIdx.x * 256 + threadIdx.x; i < n; i += gridDim.x * 256) flags[i] = 0u;
}

// Stream-K workspace of gemm_run_no_alloc, one copy per GPU for the life of
// the process: the flag area (flags and error word), then partial-sum slots.
// Host code never passes this name to a kernel or a copy: it stands for a
// host-side shadow there.  The device address comes from
// hipGetSymbolAddress, once per device (scratch_address below).
static __device__ __align__(256) char scratch[GEMM_NO_ALLOC_SCRATCH_BYTES];

namespace {

// Stream-K workspace layout: SK_MAX_WG flags, the sticky error word (padded
// to 256 bytes), then one BM*BN fp32 slot per workgroup.
constexpr int SK_MAX_WG = 4096;
constexpr int SK_FLAG_WORDS = SK_MAX_WG + 64;
constexpr size_t SK_FLAG_BYTES = SK_FLAG_WORDS * sizeof(unsigned);
// Default bound on a finisher's wait, in polls of about 100 ns per
// contributor: far beyond any wait a resident contributor needs.
constexpr int SK_SPIN_DEFAULT = 1 << 20;
static_assert(GEMM_NO_ALLOC_SCRATCH_BYTES > SK_FLAG_BYTES &&
                  GEMM_NO_ALLOC_SCRATCH_BYTES % 256 == 0,
              "no-alloc scratch holds the flag area and whole slots");

const std::vector<Variant>& table()
{
    static const std::vector<Variant> t = [] {
        std::vector<Variant> v;
        for (auto get : {bf16_variant_table, f32mfma_variant_table, f32fma_variant_table,
                         bf16dma_variant_table, f32dma_variant_table,
                         bf16dma_sweep_variant_table, bf16dma_sweep128_variant_table,
                         f32dma_sweep_variant_table,
                         bf16dma_tile_variant_table, bf16dma_192_variant_table,
                         small_variant_table}) {
            int n = 0;
            const Variant* t = get(&n);
            v.insert(v.end(), t, t + n);
        }
        return v;
    }();
    return t;
}

int find_variant(const char* name)
{
    const auto& t = table();
    for (size_t i = 0; i < t.size(); ++i)
        if (std::strcmp(t[i].name, name) == 0) return (int)i;
    return -1;
}

// Per-device caches are indexed by device ordinal; devices beyond this many
// are answered without caching.
constexpr int MAX_DEVICES = 64;
constexpr int MAX_VARIANTS = 128;

// Planning model set by gemm_set_planning_model: a compute-unit count and
// per-variant data-parallel occupancies that replace the device queries in
// the planner (0: use the query).
std::atomic<int> g_model_cus{0};
std::atomic<int> g_model_occ[MAX_VARIANTS];

// Ordinal of the current device, or -1 when it cannot be queried.
int current_device()
{
    int dev = -1;
    if (hipGetDevice(&dev) != hipSuccess) return -1;
    return dev;
}

}  // namespace

// Compute units of the current device (cached per device; entry points may
// be called from several threads at once, so the cache is atomic and a
// value is only ever replaced by the same value).
int device_cus()
{
    const int model = g_model_cus.load(std::memory_order_relaxed);
    if (model > 0) return model;
    static std::atomic<int> cached[MAX_DEVICES];
    const int dev = current_device();
    if (dev < 0) return 256;
    int n = dev < MAX_DEVICES ? cached[dev].load(std::memory_order_relaxed) : 0;
    if (n == 0) {
        if (hipDeviceGetAttribute(&n, hipDeviceAttributeMultiprocessorCount, dev) != hipSuccess ||
            n <= 0)
            n = 256;
        if (dev < MAX_DEVICES) cached[dev].store(n, std::memory_order_relaxed);
    }
    return n;
}

namespace {

// Per-shape selection.  Large tiles give the most reuse per LDS byte
// (the tile's input intensity grows with BM*BN/(BM+BN), "GEMM on NVIDIA
// GPUs", section 3) but fewer workgroups; a problem whose 256x256 tiles
// would fill less than three quarters of one wave over the compute units
// takes the 128x128 tile instead, so that more of them get work (section 5
// on tails and small shapes).  The direct-to-LDS kernels take every call
// whose operands are element-aligned and whose panel offsets fit in 32 bits;
// the register-staged kernels take the rest.  The direct-to-LDS variants
// chosen place their barrier before the last fragment step of a K-step:
// three 32-deep stages for bf16 256x256 tiles (measured 8-10 % faster than
// the half-way barrier with four stages on 8192^3 with k-contiguous A), four
// for bf16 128x128 tiles (2-5 % faster than three on six shapes from 2048^3
// to 8192x4096x1792, same occupancy of 2), and two 32-deep stages for fp32
// (1 % faster than three 16-deep ones on 4096^3).
// The direct-to-LDS variant with 256x256 (big) or 128x128 tiles for a dtype.
int dma_variant(int dtype, bool big)
{
    static const int ids[2][2] = {
        {find_variant("f32_dma32x32x2_128x128x16_w2x2_s3_late"),
         find_variant("f32_dma32x32x2_256x256x32_w2x2_s2_late")},
        {find_variant("bf16_dma32x32x16_128x128x32_w2x2_s4_late"),
         find_variant("bf16_dma32x32x16_256x256x32_w2x4_s3_late")}};
    return ids[dtype == GEMM_DTYPE_BF16_F32][big];
}

int select_variant(int dtype, int64_t M, int64_t N, int64_t /*K*/, bool dma)
{
    const int bf16_dma_big = dma_variant(GEMM_DTYPE_BF16_F32, true);
    const int bf16_dma_mid = dma_variant(GEMM_DTYPE_BF16_F32, false);
    static const int bf16_big = find_variant("bf16_mfma32x32x16_256x256x64_w2x2");
    static const int bf16_mid = find_variant("bf16_mfma16x16x32_128x128x64_w2x2");
    static const int f32_big = find_variant("f32_mfma32x32x2_256x256x32_w2x2");
    static const int f32_mid = find_variant("f32_mfma32x32x2_128x128x32_w2x2");
    const int f32_dma_big = dma_variant(GEMM_DTYPE_F32, true);
    const int f32_dma_mid = dma_variant(GEMM_DTYPE_F32, false);
    const int64_t big_tiles = ceil_div(M, 256) * ceil_div(N, 256);
    const bool big = 4 * big_tiles >= 3 * (int64_t)device_cus();
    if (dtype == GEMM_DTYPE_BF16_F32) {
        if (dma) return big ? bf16_dma_big : bf16_dma_mid;
        return big ? bf16_big : bf16_mid;
    }
    if (dma) return big ? f32_dma_big : f32_dma_mid;
    return big ? f32_big : f32_mid;
}

// Time of one K-step of a tile of variant v for a workgroup alone on a
// compute unit, in microseconds: measured on MI355X for 256x256x32 steps
// (bf16 0.85 us with 3 steps of lookahead, fp32 7.3 us with 2; 8192^3 and
// 4096^3 runs), scaled by the step's FLOPs for other tiles (128x128x32 bf16
// measured 0.245 us) and by the pipeline efficiency d/(d + kappa) of the
// variant's lookahead d relative to the measured one ("High-Performance FP16
// GEMM on NVIDIA Ada Lovelace", methodology: efficiency S/(S + kappa)).
// kappa was fitted to the sweep of every direct-to-LDS variant on MI355X:
// 0.85 steps for bf16 (1.23-1.27 before the fragment-address rework raised
// the occupancy of several 128x128 variants); 0 for fp32, whose long steps
// hide the copies at any depth.  (The occupancy part of that model is
// data_parallel_us's share.)
double step_us(const Variant& v)
{
    const bool bf16 = v.dtype == GEMM_DTYPE_BF16_F32;
    const double base = bf16 ? 0.85 : 7.3;
    const double kappa = bf16 ? 0.85 : 0.0, d_ref = bf16 ? 3.0 : 2.0;
    const double d = std::max(1, v.ahead);
    const double eff = (d / (d + kappa)) / (d_ref / (d_ref + kappa));
    return base * ((double)v.bm * v.bn * v.bk) / (256.0 * 256.0 * 32.0) / eff;
}

// Workgroups per compute unit of v's stream-K kernel (sk = true) or of its
// data-parallel kernel, from the HIP occupancy query (cached per device and
// variant, atomically as for device_cus).
int variant_occupancy(const Variant& v, bool sk = true)
{
    static std::atomic<int> cache[MAX_DEVICES][2][MAX_VARIANTS];
    const int vid = (int)(&v - table().data());
    if (!sk && vid >= 0 && vid < MAX_VARIANTS) {
        const int model = g_model_occ[vid].load(std::memory_order_relaxed);
        if (model > 0) return model;
    }
    const OccFn f = sk ? v.sk_occ : v.occ;
    if (!f) return v.bm * v.bn >= 256 * 256 ? 1 : 2;
    const int dev = current_device();
    const bool cacheable = dev >= 0 && dev < MAX_DEVICES && vid >= 0 && vid < MAX_VARIANTS;
    int n = cacheable ? cache[dev][sk][vid].load(std::memory_order_relaxed) : 0;
    if (n == 0) {
        n = std::max(1, f());
        if (cacheable) cache[dev][sk][vid].store(n, std::memory_order_relaxed);
    }
    return n;
}

// Estimated time of the data-parallel launch: waves of concurrently resident
// tiles, each K-step slowed by the workgroups sharing its compute unit.
double data_parallel_us(const Variant& v, int64_t M, int64_t N, int64_t K)
{
    const int64_t cus = device_cus(), occ = variant_occupancy(v, false);
    const int64_t tiles = ceil_div(M, v.bm) * ceil_div(N, v.bn);
    const int64_t waves = ceil_div(tiles, cus * occ);
    const double share = std::min<double>((double)occ, std::max(1.0, (double)tiles / cus));
    return waves * ceil_div(K, v.bk) * step_us(v) * share;
}

// Stream-K plan for a direct-to-LDS variant: the number of workgroups to
// split the (tile, K-step) iterations over, or 0 for data-parallel tiles.
// Stream-K divides the work evenly but pays a fix-up ("GEMM on NVIDIA GPUs",
// section 5): every workgroup that ends inside a tile writes a BM x BN fp32
// partial that the tile's finisher reads back (device-scope traffic, taken
// at 3 TB/s), and a finisher reduces its contributors one after another (one
// memory round trip, ~1.5 us, per fragment row and contributor).  Candidate
// grids: every resident workgroup slot when there are fewer slots than two
// per tile (each workgroup then spans more than a tile; the kernel takes at
// most two tiles' worth, so never fewer than half the tiles), and 2, 4, 8,
// ... workgroups per tile up to the slots.  Workgroups sharing a compute
// unit share its matrix cores.  Mode 1 takes the best candidate regardless,
// automatic mode only when it beats the data-parallel estimate `dp_us` by a
// fifth.
int stream_k_grid(const Variant& v, int64_t M, int64_t N, int64_t K, int mode, size_t ws_bytes,
                  double dp_us, double* est_us = nullptr)
{
    if (mode == 0 || !v.sk_occ || ws_bytes == 0) return 0;
    const int64_t cus = device_cus();
    const int64_t slots = std::min<int64_t>(cus * variant_occupancy(v), SK_MAX_WG);
    const int64_t tiles = ceil_div(M, v.bm) * ceil_div(N, v.bn);
    const int64_t nk = ceil_div(K, v.bk);
    const int64_t W = tiles * nk;
    const double tile_bytes = (double)v.bm * v.bn * sizeof(float);
    const int mf = v.bm / 2 / 32;  // fragment rows per wave (2x2 waves, 32-row fragments)
    int64_t cand[24];
    int nc = 0;
    // Every workgroup of a stream-K grid must be resident at once (a finisher
    // waits for lower-numbered workgroups), so the grid never exceeds the
    // slots; a range spans at most two tiles' worth of iterations, so it is
    // never below half the tiles.
    if (slots < 2 * tiles && ceil_div(tiles, 2) <= slots) cand[nc++] = slots;
    for (int64_t g = 2 * tiles; g <= slots && nc < 24; g *= 2) cand[nc++] = g;
    int64_t best_g = 0;
    double best_us = 0.0;
    for (int i = 0; i < nc; ++i) {
        const int64_t gg = std::min<int64_t>(cand[i], W / 4);
        // each workgroup's range within two tiles' worth of iterations
        if (gg < 2 || gg > SK_MAX_WG || gg > slots || !sk_grid_ok(W, gg, nk)) continue;
        const size_t need = SK_FLAG_BYTES + (size_t)gg * v.bm * v.bn * sizeof(float);
        if (need > ws_bytes) continue;
        const int64_t per = ceil_div(W, gg);
        // workgroups meeting one tile, and partial sums written and read back
        const int64_t splits = gg >= tiles ? ceil_div(nk, W / gg) : 2;
        const double contrib = (double)(gg >= tiles ? gg - tiles : gg - 1);
        // rounds of resident workgroups, each sharing its compute unit
        const double rounds = (double)ceil_div(gg, slots);
        const double share = std::max(1.0, (double)std::min(gg, slots) / cus);
        const double us = rounds * per * step_us(v) * share +
                          2.0 * contrib * tile_bytes / 3e12 * 1e6 + (double)(splits - 1) * mf * 1.5 +
                          5.0;
        if (best_g == 0 || us < best_us) {
            best_g = gg;
            best_us = us;
        }
    }
    if (best_g == 0) return 0;
    if (mode < 0 && !(best_us < 0.8 * dp_us)) return 0;
    if (est_us) *est_us = best_us;
    return (int)best_g;
}

// The direct-to-LDS kernels address a workgroup's operand panel with 32-bit
// byte offsets from the panel start: a k-contiguous panel spans (rows-1) rows
// of ld plus K elements (plus one step of overhang), an mn-contiguous one K-1
// rows of ld plus its width.  Both must stay below 2^32.
bool dma_offsets_fit(const Variant& v, bool a_kc, bool b_kc, int64_t K, int64_t lda,
                     int64_t ldb, int64_t es)
{
    const int64_t kk = K + v.bk;
    const int64_t span_a = a_kc ? (v.bm - 1) * lda + kk : kk * lda + v.bm;
    const int64_t span_b = b_kc ? (v.bn - 1) * ldb + kk : kk * ldb + v.bn;
    const int64_t lim = ((int64_t)1 << 32) - 64;
    return span_a * es < lim && span_b * es < lim;
}

// Device address of each device's copy of `scratch` (null until set up).
std::atomic<void*> scratch_addr[MAX_DEVICES];

// The current device's copy of `scratch`: its address is looked up, and its
// flag area (flags and error word) cleared by a kernel on `stream`, on the
// first call on each device.  Null if the lookup or the clearing launch
// fails.
void* scratch_address(hipStream_t stream)
{
    static std::mutex init;
    const int dev = current_device();
    if (dev < 0 || dev >= MAX_DEVICES) return nullptr;
    void* p = scratch_addr[dev].load(std::memory_order_acquire);
    if (p) return p;
    std::lock_guard<std::mutex> lock(init);
    p = scratch_addr[dev].load(std::memory_order_acquire);
    if (p) return p;
    void* dp = nullptr;
    if (hipGetSymbolAddress(&dp, HIP_SYMBOL(scratch)) != hipSuccess || !dp) return nullptr;
    unsigned* flags = static_cast<unsigned*>(dp);
    int n = SK_FLAG_WORDS;
    void* kargs[] = {&flags, &n};
    if (hipLaunchKernel(reinterpret_cast<const void*>(&clear_flags_kernel), dim3(16), dim3(256),
                        kargs, 0, stream) != hipSuccess)
        return nullptr;
    scratch_addr[dev].store(dp, std::memory_order_release);
    return dp;
}

// Read a stream-K workspace's error word after `stream` drains; when it is
// set, clear the flag area on `stream` and report GEMM_ERR_STREAM_K.
gemm_status_t check_and_clear(void* ws, hipStream_t stream)
{
    unsigned err = 0;
    const unsigned* word = static_cast<const unsigned*>(ws) + SK_MAX_WG;
    if (hipMemcpyAsync(&err, word, sizeof(err), hipMemcpyDeviceToHost, stream) != hipSuccess ||
        hipStreamSynchronize(stream) != hipSuccess)
        return GEMM_ERR_HIP;
    if (err == 0) return GEMM_OK;
    // a finisher gave up: contributors it did not wait for may have raised
    // their flags after it; clear every flag and the error word
    unsigned* flags = static_cast<unsigned*>(ws);
    int n = SK_FLAG_WORDS;
    void* kargs[] = {&flags, &n};
    if (hipLaunchKernel(reinterpret_cast<const void*>(&clear_flags_kernel), dim3(16), dim3(256),
                        kargs, 0, stream) != hipSuccess ||
        hipStreamSynchronize(stream) != hipSuccess)
        return GEMM_ERR_HIP;
    return GEMM_ERR_STREAM_K;
}

// What a call looks like to the kernel choice.
struct CallDesc {
    int dtype;          // gemm_dtype_t
    bool a_kc, b_kc;    // A with transA == N, B with transB == T
    int64_t M, N, K, lda, ldb;
    bool epi;           // a fused epilogue with something to do
    bool wide;          // A and B element-aligned (16-byte accesses allowed)
    bool rows16;        // every row of A and B starts 16-byte aligned
    int forced;         // forced variant, or -1
    int sk_mode;        // stream-K policy (-1 automatic, 0 never, 1 when allowed)
    size_t ws_bytes;    // stream-K workspace bytes (0: none)
};

// The choice for one call: the variant, stream-K grid (0: whole tiles),
// whether the direct-to-LDS kernel's 16-byte path applies, whether a bf16 NN
// call runs as D^T = B^T A^T, and the launch tables it needs.
struct Plan {
    int id = -1;
    int sk = 0;
    bool aligned = false;
    bool nn_t = false;
    const LaunchFn (*sk_fn)[2] = nullptr;
    const EpiFns* ef = nullptr;
};

// Stream-K launch functions of a variant for a call's output type and
// epilogue (null: the variant has none, so whole tiles).
const LaunchFn (*sk_launchers(const Variant& x, int op_dtype, bool out_bf16, bool epi))[2]
{
    if (x.kind != KIND_MFMA_DMA || !x.sk_occ) return nullptr;
    if (!out_bf16 && !epi) return x.sk_fn;
    if (x.bm != 256 && x.bm != 128) return nullptr;
    if (&x != &table()[dma_variant(op_dtype, x.bm == 256)]) return nullptr;
    const SkFns* f = nullptr;
    if (op_dtype == GEMM_DTYPE_F32) {
        f = epi ? sk_fns_f32(x.bm) : nullptr;
    } else {
        const int kind = !epi ? 0 : out_bf16 ? 2 : 1;
        f = x.bm == 256 ? sk_fns_bf16_256(kind) : sk_fns_bf16_128(kind);
    }
    return f ? f->fn : nullptr;
}

// Fused-epilogue launches of variant `id` for the call's operand and output
// types, or null where the variant carries none (the selected square
// direct-to-LDS variants, the non-square bf16 tiles and the 2-stage and
// paired 128x128 bf16 rings do).
const EpiFns* epi_fns_for(int id, int op_dtype, bool out_bf16)
{
    if (id < 0) return nullptr;
    const Variant& v = table()[id];
    if (id == dma_variant(op_dtype, v.bm == 256))
        return op_dtype == GEMM_DTYPE_F32 ? epi_fns_f32(v.bm)
               : out_bf16                 ? epi_fns_bf16_out(v.bm)
                                          : epi_fns_bf16(v.bm);
    if (op_dtype != GEMM_DTYPE_BF16_F32) return nullptr;
    static const int tiles[6] = {find_variant("bf16_dma32x32x16_128x256x32_w2x2_s3_late"),
                                 find_variant("bf16_dma32x32x16_192x256x32_w2x4_s3_late"),
                                 find_variant("bf16_dma32x32x16_256x192x32_w4x2_s3_late"),
                                 find_variant("bf16_dma32x32x16_128x128x32_w2x2_s2_late"),
                                 find_variant("bf16_dma32x32x16_128x128x32_w2x2_s4_late_pair"),
                                 find_variant("bf16_dma32x32x16_128x128x64_w2x2_s3_late")};
    for (int w = 0; w < 6; ++w)
        if (id == tiles[w]) return out_bf16 ? epi_fns_tile_bf16out(w) : epi_fns_tile_f32out(w);
    return nullptr;
}

// The whole host choice for a call, shared by gemm_run and
// gemm_select_variant.  Returns GEMM_OK or why the call cannot run.
gemm_status_t plan_call(const CallDesc& c, Plan& pl)
{
    const int op_dtype = c.dtype == GEMM_DTYPE_F32 ? GEMM_DTYPE_F32 : GEMM_DTYPE_BF16_F32;
    const bool out_bf16 = c.dtype == GEMM_DTYPE_BF16_BF16;
    const int64_t es = op_dtype == GEMM_DTYPE_F32 ? 4 : 2;
    const int64_t M = c.M, N = c.N, K = c.K;
    int id = c.forced;
    // Small problems: where 128x128 tiles would occupy at most a sixteenth of
    // the compute units (256^3: 4 tiles), one 16x16 block per workgroup
    // spreads the output over them (fp32 256^3 measured 19.5 us on four
    // 128x128 tiles).  Not when stream-K is forced, nor for bf16 output or a
    // fused epilogue, which the small kernel does not carry.
    if (id < 0 && !c.epi && !out_bf16 && c.sk_mode != 1 && K <= 4096 &&
        16 * ceil_div(M, 128) * ceil_div(N, 128) <= (int64_t)device_cus()) {
        static const int small[2] = {find_variant("f32_small16x16x16_w4"),
                                     find_variant("bf16_small16x16x32_w4")};
        if (small[op_dtype] >= 0) {
            pl.id = small[op_dtype];
            pl.sk = 0;
            pl.aligned = c.wide;
            return GEMM_OK;
        }
    }
    if (id < 0) {
        const Variant& big = table()[select_variant(op_dtype, M, N, K, true)];
        id = select_variant(op_dtype, M, N, K,
                            c.wide && dma_offsets_fit(big, c.a_kc, c.b_kc, K, c.lda, c.ldb, es));
    }
    // fp32 from 3/4 of a wave of 256x256 tiles: 128x128 tiles (three
    // workgroups per compute unit) for K <= 1024, where they were the fastest
    // candidate on every shape timed (the D write weighs more and three
    // resident workgroups spread it), and for longer K where the
    // data-parallel model gives them less time, i.e. where the 256x256
    // tiles' last wave would be partly empty while the 128x128 rounds come
    // out fuller.  Every fp32 whole-tile candidate timed on 36 shapes (M, N
    // in 1024 .. 8192) per K and layout (TN, NT; ms, one box, 256x256 ->
    // 128x128): TN 6144^2 x 4096 2.79 -> 2.09 (576 tiles, the third wave
    // 1/4 full), TN 3072x6144x256 0.137 -> 0.084, TN 8192x3072x1024 0.480
    // -> 0.366; at long K the model keeps 256x256 on whole waves (4096^3:
    // 0.933 against 0.932 on 128x128; 8192^2 x 4096).  Mean ratio to the
    // fastest candidate 1.140 -> 1.000 at K = 256 and 1.052 -> 1.000 at 1024
    // (128x128 fastest on all 144 shapes), 1.011 -> 1.001 at 4096 (the
    // model's choices), judged on one run.
    if (c.forced < 0 && op_dtype == GEMM_DTYPE_F32 && id == dma_variant(GEMM_DTYPE_F32, true)) {
        const int mid = dma_variant(GEMM_DTYPE_F32, false);
        if (mid >= 0 && dma_offsets_fit(table()[mid], c.a_kc, c.b_kc, K, c.lda, c.ldb, es) &&
            (K <= 1024 ||
             data_parallel_us(table()[mid], M, N, K) < data_parallel_us(table()[id], M, N, K)))
            id = mid;
    }
    const Variant& v = table()[id];
    if (v.dtype != op_dtype) return GEMM_ERR_NOT_SUPPORTED;
    // bf16 C/D: only the selected direct-to-LDS variants carry that epilogue,
    // for element-aligned operands whose panel offsets fit in 32 bits
    if (out_bf16 && !v.bo_nn_t_fn) return GEMM_ERR_NOT_SUPPORTED;
    // a direct-to-LDS kernel whose offsets would overflow stages every step
    // through registers instead (its ALIGNED == false instantiation)
    const bool aligned =
        c.wide && (v.kind != KIND_MFMA_DMA || dma_offsets_fit(v, c.a_kc, c.b_kc, K, c.lda, c.ldb, es));
    const double dp_us = data_parallel_us(v, M, N, K);
    double sk_us = 0.0;
    int sk = (aligned && sk_launchers(v, op_dtype, out_bf16, c.epi))
                 ? stream_k_grid(v, M, N, K, c.sk_mode, c.ws_bytes, dp_us, &sk_us)
                 : 0;
    // bf16 operands (fp32 or bf16 output, with or without the fused
    // epilogue), at most half a wave of 128x128 tiles, K >= 3072: stream-K
    // wherever a grid fits.  With one tile per busy compute unit the
    // whole-tile kernel is bound by each K-step's copy latency, more so with
    // a k-contiguous operand (NN 1024^2 x 4096 0.0320 ms against 0.0255 for
    // TN), and the model above, which needs a fifth's margin, declined grids
    // that were faster.  Every such
    // shape timed (M, N in 512 .. 2048, 48 to 128 tiles, K = 3072, 4096,
    // 6144, all four layouts; one box, ms, whole tiles -> stream-K): with a
    // k-contiguous operand 0.58-0.90 (NN 1024^2 x 4096 0.0320 -> 0.0231), TN
    // 0.66-0.93 up to 96 tiles (1024^2 x 4096 0.0255 -> 0.0208); TN at 128
    // tiles only from K = 6144 (0.84-0.88; at K = 3072 up to 1.15 with bf16
    // output).  At K = 2048 it was mixed (0.76-1.36), from 144 tiles it lost
    // or about tied (0.95-1.41; TN 1536^2 x 4096 0.0270 -> 0.0327).  With
    // bias + GELU fused, TN and NN: 0.65-1.00 where this takes it.
    if (sk == 0 && c.forced < 0 && c.sk_mode < 0 && aligned && op_dtype == GEMM_DTYPE_BF16_F32 &&
        v.kind == KIND_MFMA_DMA && v.bm == 128 && v.bn == 128 && K >= 3072 &&
        sk_launchers(v, op_dtype, out_bf16, c.epi)) {
        const int64_t t128 = ceil_div(M, 128) * ceil_div(N, 128), cus = device_cus();
        if (2 * t128 <= cus && (c.a_kc || c.b_kc || 8 * t128 <= 3 * cus || K >= 6144)) {
            // Both operands k-contiguous (NT), fp32 output, aligned rows: the
            // stream-K launch of the 64-deep variant, whose copied rows are
            // whole 128-byte lines for both operands.  Against the 4-stage
            // ring's stream-K, three runs on three boxes: NT 0.78-1.05, means
            // 0.91-0.94 (512x2048x3072 0.0245 -> 0.0194 ms); with one
            // k-contiguous operand (NN, TT) 0.89-1.14, mean 1.00, and TN
            // 1.04-1.15, so those keep the 4-stage ring.
            static const int deep = find_variant("bf16_dma32x32x16_128x128x64_w2x2_s3_late");
            double d_us = 0.0;
            const int sk_d =
                (deep >= 0 && c.a_kc && c.b_kc && c.rows16 && !out_bf16 && !c.epi &&
                 sk_launchers(table()[deep], op_dtype, out_bf16, c.epi) &&
                 dma_offsets_fit(table()[deep], c.a_kc, c.b_kc, K, c.lda, c.ldb, es))
                    ? stream_k_grid(table()[deep], M, N, K, 1, c.ws_bytes, dp_us, &d_us)
                    : 0;
            if (sk_d > 0) {
                id = deep;
                sk = sk_d;
                sk_us = d_us;
            } else {
                sk = stream_k_grid(v, M, N, K, 1, c.ws_bytes, dp_us, &sk_us);
            }
        }
    }
    // bf16, fp32 output, 3/8 to 1/2 of a wave of 256x256 tiles and a very
    // long K (NT from K = 8192, other layouts from 16384, e.g. weight
    // gradients over many tokens): stream-K on the 8-wave 256x256 kernel.
    // The whole-tile rules below take 128x256 or the paired 128x128 ring
    // there, and the model rejected the 256x256 grid (its step time is
    // calibrated on 8192^3 at the board's power limit, where the clock sits
    // near 1.6 GHz; with a third of the units busy it runs faster).  Timed
    // on 96 and 100 tiles of 256x256 (2048x3072, 3072x2048, 2560^2,
    // 1536x4096; one box, ms, automatic -> stream-K on 256x256): NT
    // 0.87-0.95 at K = 8192 (2048x3072 0.1129 -> 0.0981) and 0.88-0.90 at
    // 16384; NN 0.91-0.96 and TN 0.93-0.96 at 16384, while at 8192 they
    // varied 0.95-1.03.  On a second box, also over 112 tiles (1792x4096,
    // 3584x2048) and in TT, against the fastest whole-tile candidate: NT
    // 0.92-1.03 at 8192 and 0.86-0.91 at 16384; NN, TN, TT 0.90-0.98 at
    // 16384.
    if (sk == 0 && c.forced < 0 && c.sk_mode < 0 && aligned && op_dtype == GEMM_DTYPE_BF16_F32 &&
        !out_bf16 && !c.epi && K >= ((c.a_kc && c.b_kc) ? 8192 : 16384)) {
        const int64_t t256 = ceil_div(M, 256) * ceil_div(N, 256), cus = device_cus();
        const int big = dma_variant(GEMM_DTYPE_BF16_F32, true);
        if (3 * cus <= 8 * t256 && 8 * t256 < 4 * cus && big >= 0 &&
            sk_launchers(table()[big], op_dtype, out_bf16, c.epi) &&
            dma_offsets_fit(table()[big], c.a_kc, c.b_kc, K, c.lda, c.ldb, es)) {
            double b_us = 0.0;
            const int sk_b = stream_k_grid(table()[big], M, N, K, 1, c.ws_bytes, dp_us, &b_us);
            if (sk_b > 0) {
                id = big;
                sk = sk_b;
                sk_us = b_us;
            }
        }
    }
    if (c.forced < 0 && aligned && v.kind == KIND_MFMA_DMA && c.sk_mode != 0) {
        // With a workspace, stream-K on the other tile size competes too; the
        // lowest estimate wins.  It has to beat that tile size's own
        // data-parallel estimate as well as the chosen one's: stream-K over
        // whole waves of tiles only adds its fix-up (fp32 4096^2 x 256 took
        // stream-K on 256 tiles of 256x256, one workgroup per tile, at 0.0737
        // ms against 0.0688 for the chosen 128x128 tiles).
        const int other = dma_variant(op_dtype, v.bm < 256);
        if (other != id && sk_launchers(table()[other], op_dtype, out_bf16, c.epi) &&
            dma_offsets_fit(table()[other], c.a_kc, c.b_kc, K, c.lda, c.ldb, es)) {
            double o_us = 0.0;
            const double ref_us = std::min(dp_us, data_parallel_us(table()[other], M, N, K));
            const int sk_o =
                stream_k_grid(table()[other], M, N, K, c.sk_mode, c.ws_bytes, ref_us, &o_us);
            if (sk_o > 0 && (sk == 0 || o_us < sk_us)) {
                id = other;
                sk = sk_o;
            }
        }
    }
    // bf16 operands, whole tiles, fp32 output (bf16 output too where the
    // variant carries it): tile shapes beyond the two square ones, from
    // measurements on MI355X with fp32 output (us, one box, automatic
    // choice before -> after):
    //  * K <= 1024 with at least a full wave of 256x256 tiles: 128x256 tiles,
    //    two workgroups per compute unit, so one's prologue and epilogue hide
    //    behind the other's matrix work (8192x4096x512 56.8 -> 46.2,
    //    16384x4096x512 119 -> 95, 8192^2 x 512 111 -> 87).
    //  * Fewer 256x256 tiles than three quarters of a wave, K >= 2048, and
    //    128x256 tiles that fill between three quarters of a wave and one
    //    per compute unit: 128x256 (4096x2048x4096 66.9 -> 62.6, 2560^2 x
    //    4096 57.7 -> 55.5).
    //  * Otherwise, at least half a wave of 256x256 tiles and a long K, or
    //    rows that are not 16-byte aligned (every 16-byte copy then
    //    straddles two units, and two waves per SIMD hide that latency): the
    //    8-wave 256x256 kernel (3072^3 76.5 -> 58.6; 4093x2051x1537 A^T B
    //    58.5 -> 50.1).
    bool untransposed = false;  // an NN call that keeps its orientation
    bool keep_depth = false;    // the 128x128 rings keep their 4-stage depth
    // a variant serves the call's output type and epilogue (bf16 output and
    // the fused epilogue: launches of its own)
    auto serves = [&](const Variant& x) {
        return (!out_bf16 || x.bo_nn_t_fn != nullptr) &&
               (!c.epi || epi_fns_for((int)(&x - table().data()), op_dtype, out_bf16) != nullptr);
    };
    if (sk == 0 && c.forced < 0 && aligned && op_dtype == GEMM_DTYPE_BF16_F32) {
        static const int wide_tile = find_variant("bf16_dma32x32x16_128x256x32_w2x2_s3_late");
        const int64_t cus = device_cus();
        const int64_t t256 = ceil_div(M, 256) * ceil_div(N, 256);
        const int64_t t12 = ceil_div(M, 128) * ceil_div(N, 256);
        const int big_id = dma_variant(GEMM_DTYPE_BF16_F32, true);
        const bool wide_ok = wide_tile >= 0 && serves(table()[wide_tile]) &&
                             dma_offsets_fit(table()[wide_tile], c.a_kc, c.b_kc, K, c.lda, c.ldb, es);
        // (with bf16 output, whose stores weigh half as much, only from four
        // waves of 256x256 tiles: 8192x4096x512 0.0433 -> 0.0446 ms on
        // 128x256 tiles, 16384x4096x512 0.0795 -> 0.0761).  Both operands
        // k-contiguous (NT): 128x256 copies them half a line per step while
        // the square tiles pair the copies, so 128x256 only for K <= 512
        // (NT 8192x4096x1024 0.0766 vs 0.0742 ms on 256x256, 8192x2048x1024
        // 0.0409 vs 0.0375), none of the long-K rule (the paired 128x128
        // ring wins: NT 4096x2048x4096 0.0710 vs 0.0660, 8192x1024x4096
        // 0.0699 vs 0.0647), and 256x256 (or, below, a 192-wide tile) from
        // more than half a wave of 256x256 tiles and K >= 1024 (NT 3072^2 x
        // 1024 0.0305 on 128x128 vs 0.0261 on 256x192).
        const bool both_kc = c.a_kc && c.b_kc;
        const bool big_fits = dma_offsets_fit(table()[big_id], c.a_kc, c.b_kc, K, c.lda, c.ldb, es);
        // Short K, fp32 output (the D write is most of the traffic): 128x256
        // tiles only where their rounds at two per compute unit come out
        // nearly whole (at least 9/10 full for K <= 256, 3/4 for K <= 512),
        // the 128x128 rings elsewhere from three quarters of a wave of
        // 256x256 tiles; and with both operands k-contiguous and K below
        // 1024, the 128x128 rings (paired) over more than a wave of 256x256
        // tiles whose last wave is less than 9/10 full.  From every whole-tile
        // candidate timed on 36 shapes (M, N in 1024 .. 8192) per K and layout
        // (TN, NT; ms, one box, automatic choice before -> 128x128 rings):
        // TN 6144x3072x256 0.0261 (128x256; 288 tiles of 256x256, so its
        // rounds are 9/16 full) -> 0.0206-0.0222, TN 3072x4096x256 0.0169
        // (256x256, 192 tiles) -> 0.0145-0.0152, NT 6144x2048x512 0.0217 ->
        // 0.0193 (paired), NT 6144x3072x768 0.0520 (256x256) -> 0.0413
        // (paired); mean ratio to the fastest candidate 1.066 -> 1.038 at
        // K = 256, 1.034 -> 1.026 at 512, 1.040 -> 1.027 at 768.
        const auto rounds_at_least = [&](int64_t tiles, int64_t per_cu, int num, int den) {
            const int64_t slots = per_cu * cus;
            return den * tiles >= num * ceil_div(tiles, slots) * slots;
        };
        const int mid_id = dma_variant(GEMM_DTYPE_BF16_F32, false);
        const bool mid_ok = serves(table()[mid_id]) &&
                            dma_offsets_fit(table()[mid_id], c.a_kc, c.b_kc, K, c.lda, c.ldb, es);
        // (measured with fp32 output and 16-byte aligned rows; other calls
        // keep the rules below)
        const bool measured = !out_bf16 && c.rows16;
        // bf16 output, K <= 512, aligned rows, from 3/4 to 4 waves of 256x256
        // tiles (half the D bytes, so the matrix work weighs more): 256x256
        // where its waves are whole, below one wave the 192-wide search that
        // follows; otherwise 128x256 where its rounds at two per compute unit
        // are at least 3/4 full, else the 128x128 ring.  Same grid with bf16
        // D (ms, one box, 256x256 -> the rule's choice): TN 6144x3072x256
        // 0.0259 -> 0.0209 (128x128), TN 3072x4096x256 0.0142 -> 0.0124
        // (192x256), TN 8192x3072x512 0.0366 -> 0.0320 (128x256); mean ratio
        // to the fastest candidate 1.061 -> 1.015 at K = 256, 1.045 -> 1.013
        // at 512 (fitted to that run).
        const bool short_bo = out_bf16 && c.rows16 && K <= 512;
        const bool wide_rounds = K > 512 || !measured ||
                                 rounds_at_least(t12, 2, K <= 256 ? 9 : 3, K <= 256 ? 10 : 4);
        // Only B k-contiguous (A^T B^T): the 128x256 tile puts its 256-wide
        // side on that operand, copying 256 rows half a line per step; the
        // 256x128 tile puts 128 there.  From the same grid (TT, fp32 output):
        // at 512 < K <= 1024 over a wave of 256x256 tiles the 256x128 tile
        // (3072x8192x1024 0.0572 ms against 0.0540), and 256x128 instead of
        // 128x256 in the long-K rule below (4096x2048x4096 0.0676 against
        // 0.0587); mean ratio to the fastest candidate 1.039 -> 1.009 at K =
        // 1024, 1.029 -> 1.004 at 4096 (on a second run).  At K <= 512 only
        // over 3/4 to 1 wave of 256x256 tiles (below); elsewhere the rules
        // above (a rule sending more of these calls to the 128x128 rings won
        // some shapes on one run and lost them on the next).
        static const int tall_tile = find_variant("bf16_dma32x32x16_256x128x32_w2x2_s3_late");
        const bool b_only_kc = c.b_kc && !c.a_kc;
        const bool tall_ok = measured && b_only_kc && tall_tile >= 0 &&
                             serves(table()[tall_tile]) &&
                             dma_offsets_fit(table()[tall_tile], c.a_kc, c.b_kc, K, c.lda, c.ldb, es);
        // Rows not 16-byte aligned (every 16-byte copy straddles two units),
        // fp32 output, K <= 512: no 128x256 tiles, which lost 16-33 % there;
        // with a k-contiguous operand (NN, NT, TT) 256x256 tiles over waves
        // at least 3/4 full (NN runs as stored, below), everything else the
        // 128x128 rings (NT 8189x4093x511 0.0906 on the paired 128x128 ring
        // -> 0.0798 on 256x256, on a second grid run; at 288 tiles of 256x256
        // the 2-stage 128x128 ring was fastest in every layout).  From
        // every whole-tile candidate on 36 shapes with odd sides (1021 ..
        // 8189) per layout, K = 511 (ms, one box): TN 4093x4093 0.0513 on
        // 128x256 -> 0.0393 on the 4-stage 128x128 ring, NN 4093x4093 0.0536
        // -> 0.0412 on 256x256 as stored; mean ratio to the fastest candidate
        // 1.126 -> 1.020 (TN), 1.140 -> 1.026 (NN), fitted to that run.
        const bool mis_short = !out_bf16 && !c.rows16 && K <= 512;
        // bf16 output, no k-contiguous operand, K <= 256, from 3/8 of a wave
        // of 256x256 tiles: the 2-stage 128x128 ring (three workgroups per
        // compute unit), the fastest candidate on 22 of 28 such grid shapes
        // and within 6 % on the rest (TN 4096x3072x256 0.0142 ms on 256x192
        // -> 0.0123, 6144x6144x256 0.0349 on 128x256 -> 0.0309; mean ratio
        // to the fastest candidate 1.074 -> 1.013 on that run)
        static const int s2_id = find_variant("bf16_dma32x32x16_128x128x32_w2x2_s2_late");
        const bool s2_bo = short_bo && !c.a_kc && !c.b_kc && K <= 256 && 8 * t256 >= 3 * cus &&
                           s2_id >= 0 && serves(table()[s2_id]) &&
                           dma_offsets_fit(table()[s2_id], c.a_kc, c.b_kc, K, c.lda, c.ldb, es);
        // Three quarters to one wave of 256x256 tiles at K <= 512, fp32 output,
        // aligned rows, with B k-contiguous: the 2-stage 128x128 ring, which
        // the round model takes there (its 3 workgroups per compute unit run
        // the 128x128 tiles in one round), trailed the deeper rings, its two
        // stages too shallow for the half-line copies of a k-contiguous
        // operand.  TT (only B k-contiguous) at 256 < K <= 512 takes 256x128;
        // NT (both) at K <= 512 keeps the paired 4-stage ring.  Two grid runs
        // on two boxes (ms, 2-stage ring -> the rule's choice): TT
        // 4096x3072x512 0.0225 -> 0.0203 and 0.0207 -> 0.0183, NT
        // 6144x2048x512 0.0226 -> 0.0197 and 0.0210 -> 0.0180; mean ratio to
        // the fastest candidate over the four such shapes and two runs 1.10
        // -> 1.01 (TT, K = 512), 1.14 -> 1.02 (NT, K = 512), 1.08 -> 1.03
        // (NT, K = 256).  TN (no k-contiguous operand) and TT at K = 256 stay
        // on the 2-stage ring (mean ratio 1.03 there).
        const bool ring_wave = measured && K <= 512 && 4 * t256 >= 3 * cus && t256 < cus;
        keep_depth = ring_wave && both_kc;
        if (s2_bo) {
            id = s2_id;
        } else if (tall_ok && K > 512 && K <= 1024 && t256 >= cus) {
            id = tall_tile;
        } else if (tall_ok && ring_wave && K > 256) {
            id = tall_tile;
        } else if (mis_short) {
            if ((c.a_kc || c.b_kc) && 4 * t256 >= 3 * cus && rounds_at_least(t256, 1, 3, 4) &&
                big_fits)
                id = big_id;
            else if (mid_ok)
                id = mid_id;
        } else if (wide_ok && K <= (both_kc ? 512 : 1024) && t256 >= (out_bf16 ? 4 : 1) * cus &&
                   wide_rounds) {
            id = wide_tile;
        } else if (measured && K <= 512 && 4 * t256 >= 3 * cus && mid_ok) {
            id = mid_id;
        } else if (measured && both_kc && K < 1024 && t256 > cus &&
                   !rounds_at_least(t256, 1, 9, 10) && mid_ok) {
            id = mid_id;
        } else if (short_bo && 4 * t256 >= 3 * cus && t256 < 4 * cus) {
            if (t256 < cus || rounds_at_least(t256, 1, 9, 10)) {
                if (big_fits && serves(table()[big_id])) id = big_id;
            } else if (wide_ok && rounds_at_least(t12, 2, 3, 4)) {
                id = wide_tile;
            } else if (mid_ok) {
                id = mid_id;
            }
        } else if (4 * t256 < 3 * cus) {
            // bf16 output, aligned rows, one or no operand k-contiguous:
            // 128x256 tiles filling 3/4 to 1 of a wave from K = 1024 (with
            // bf16 D, ms, one box: TN 3072x2048x1024 0.0214 on 128x128 ->
            // 0.0188).  Both operands k-contiguous take the paired 128x128
            // ring there, as with fp32 D (NT 2048x4096x4096: 0.0667 on it
            // against 0.0740 on 128x256).
            const bool bo_wide = out_bf16 && c.rows16 && wide_ok && K >= 1024 && t12 <= cus &&
                                 4 * t12 >= 3 * cus;
            // only B k-contiguous, rows not 16-byte aligned, fp32 output:
            // 256x128 where 128x256 tiles would fill 3/4 to 1 of a wave, from
            // K = 1024 (odd-sided grid, TT: fastest candidate on all 16 such
            // shapes at K = 1537 and 4093; 2045x4093x4093 0.0941 on 128x256 ->
            // 0.0832)
            const bool tall_mis = !out_bf16 && !c.rows16 && b_only_kc && tall_tile >= 0 &&
                                  serves(table()[tall_tile]) &&
                                  dma_offsets_fit(table()[tall_tile], c.a_kc, c.b_kc, K, c.lda,
                                                  c.ldb, es);
            if (both_kc) {
                if (2 * t256 > cus && K >= 1024 && big_fits) id = big_id;
            } else if (tall_mis && K >= 1024 && t12 <= cus && 4 * t12 >= 3 * cus) {
                id = tall_tile;
            } else if (bo_wide || (wide_ok && K >= 2048 && t12 <= cus && 4 * t12 >= 3 * cus)) {
                id = tall_ok ? tall_tile : wide_tile;
            } else if (2 * t256 >= cus && (K >= 2048 || !c.rows16) && big_fits) {
                id = big_id;
            }
        }
        // Tiles with a 192-wide side (192x256, 256x192) where they fill whole
        // waves of compute units that 256x256 tiles leave partly empty: a
        // wave of them takes about 3/4 of a 256x256 wave, so they win when
        // 3/4 of their waves stays below 0.95 of the 256x256 waves.  Each
        // runs as stored or, for NN, as D^T (which swaps the sides the tile
        // dimensions lie on); the fewest waves win, and on a tie D^T for NN
        // unless rows are not 16-byte aligned.  Measured on MI355X (ms,
        // 256x256 -> 192-wide, one box per group): NN 8192x1536x4096 0.0982
        // -> 0.0910 (256 tiles instead of 192, one wave), 8192x4608x4096
        // 0.2766 -> 0.2538, 3072^3 NN 0.0576 -> 0.0551 and TN 0.0565 ->
        // 0.0532, NN 4093x2051x1537 0.0549 -> 0.0442 as stored (0.0590 as
        // D^T); NT 8192x1536x4096 0.0974 -> 0.0888 and 8192x3072x4096 0.1868
        // -> 0.1723 (256x192), NN 1536x8192x4096 0.0917 -> 0.0867.
        static const int w192[2] = {find_variant("bf16_dma32x32x16_192x256x32_w2x4_s3_late"),
                                    find_variant("bf16_dma32x32x16_256x192x32_w4x2_s3_late")};
        if (id == big_id && (K >= 1024 || (short_bo && t256 < cus))) {
            constexpr int64_t NONE = INT64_MAX / 64;
            int64_t best_w = NONE;
            bool best_pref = false;
            for (int vi = 0; vi < 2; ++vi) {
                if (w192[vi] < 0 || !serves(table()[w192[vi]])) continue;
                // 256x192 on rows that are not 16-byte aligned ran 13-46 %
                // behind the fastest candidate (odd-sided grid, K = 1537 and
                // 4093: TN 4093x6141x1537 0.1437 against 0.1076 on 256x256),
                // 192x256 where it was chosen within a few %
                if (vi == 1 && !c.rows16) continue;
                const Variant& vv = table()[w192[vi]];
                for (int tr = 0; tr < 2; ++tr) {
                    const bool ok = tr ? (c.rows16 && c.a_kc && !c.b_kc && vv.nn_t_fn &&
                                          dma_offsets_fit(vv, false, true, K, c.ldb, c.lda, es))
                                       : dma_offsets_fit(vv, c.a_kc, c.b_kc, K, c.lda, c.ldb, es);
                    if (!ok) continue;
                    const int64_t tiles = tr ? ceil_div(N, vv.bm) * ceil_div(M, vv.bn)
                                             : ceil_div(M, vv.bm) * ceil_div(N, vv.bn);
                    const int64_t w = ceil_div(tiles, cus);
                    // D^T first for aligned NN rows, as stored otherwise; then
                    // 192x256 before 256x192
                    const bool pref = (tr == 1) == c.rows16;
                    if (w < best_w || (w == best_w && pref && !best_pref)) {
                        best_w = w;
                        best_pref = pref;
                        if (15 * w < 19 * ceil_div(t256, cus)) {  // 3/4 w < 0.95 w256
                            id = w192[vi];
                            untransposed = c.a_kc && !c.b_kc && tr == 0;
                        }
                    }
                }
            }
        }
    }
    // bf16 128x128 whole tiles: the 2-stage ring fits 3 workgroups on a
    // compute unit where the 4-stage one fits 2.  The shallower ring wins
    // when that removes a round of tiles (4093x2051x1537: 544 tiles in one
    // round instead of a full round and a nearly empty one; measured 0.0593
    // vs 0.0624 ms), which the round and pipeline-depth model above decides.
    // Neither variant has a transposed-output instantiation (NN keeps its
    // orientation on them); both carry bf16 output and the fused epilogue.
    if (sk == 0 && c.forced < 0 && aligned &&
        id == dma_variant(GEMM_DTYPE_BF16_F32, false)) {
        static const int s2 = find_variant("bf16_dma32x32x16_128x128x32_w2x2_s2_late");
        if (s2 >= 0 && !keep_depth && serves(table()[s2]) &&
            data_parallel_us(table()[s2], M, N, K) < data_parallel_us(table()[id], M, N, K))
            id = s2;
        // Otherwise, with a k-contiguous operand and more tiles than compute
        // units (two workgroups on a unit hide the latency of the larger
        // copies), the 4-stage ring copying that operand two K-steps at a
        // time: measured 5-16 % faster from 324 to 544 tiles (2304^3 36.9
        // vs 44.0 us, 2560^2 x 4096 62.0 vs 72.8) and 5-22 % slower at 256
        // tiles and fewer.
        static const int pair = find_variant("bf16_dma32x32x16_128x128x32_w2x2_s4_late_pair");
        if (id != s2 && pair >= 0 && serves(table()[pair]) && (c.a_kc || c.b_kc) &&
            ceil_div(M, 128) * ceil_div(N, 128) > (int64_t)device_cus())
            id = pair;
        // One 128x128 tile per busy compute unit (more than half a wave, at
        // most one), a k-contiguous operand, K >= 3072, aligned rows: 64-deep
        // K-steps (three stages), as stored; with either output type and
        // with or without the fused epilogue.  A k-contiguous
        // row of a 32-deep bf16 step is half a 128-byte line; at 64 it is a
        // whole line, and with no second workgroup on the unit to hide the
        // copies that halves their requests per FLOP.  Timed on 63 such
        // shapes (M, N in 1024 .. 4096, 144 to 256 tiles, K = 3072, 4096,
        // 8192, NN, NT, TT; one box, ms, the 4-stage ring -> 64-deep steps):
        // 0.75-1.00 of the automatic time, mean 0.90 (NT 1536^2 x 3072 0.0313
        // -> 0.0236, NN 1536^2 x 4096 0.0344 -> 0.0295); TN, whose rows
        // along mn already copy whole lines, lost 5-16 %.  With bf16 output,
        // bias + GELU, or both (NN, NT, TT, 24 shapes each): 0.77-0.98 of
        // the 4-stage ring, means 0.89-0.90.
        static const int deep = find_variant("bf16_dma32x32x16_128x128x64_w2x2_s3_late");
        const int64_t t128 = ceil_div(M, 128) * ceil_div(N, 128), cus = device_cus();
        if (id == dma_variant(GEMM_DTYPE_BF16_F32, false) && deep >= 0 && serves(table()[deep]) &&
            c.rows16 && (c.a_kc || c.b_kc) && K >= 3072 && 2 * t128 > cus && t128 <= cus &&
            dma_offsets_fit(table()[deep], c.a_kc, c.b_kc, K, c.lda, c.ldb, es)) {
            id = deep;
            untransposed = true;
        }
    }
    const Variant& vr = table()[id];
    // bf16 NN with whole tiles: run as D^T = B^T A^T, which puts the
    // mn-contiguous operand first (measured on 8192^3, same box: TT layout
    // 1282 vs NN 1235 TFLOP/s); the transposed-output epilogue writes D.
    // (not for rows that are not 16-byte aligned: as D^T the transposed
    // epilogue writes D in short row pieces, each straddling two lines of the
    // misaligned rows; NN 8189x2045x1537 0.0683 as D^T on 256x256 against
    // 0.0605 as stored, 4093x4093x511 0.0535 against 0.0412)
    const bool nn_t = sk == 0 && c.forced < 0 && !untransposed && vr.nn_t_fn && aligned &&
                      c.rows16 && c.a_kc && !c.b_kc &&
                      dma_offsets_fit(vr, false, true, K, c.ldb, c.lda, es);
    if (out_bf16 && !aligned) return GEMM_ERR_NOT_SUPPORTED;
    // fused epilogue: only the selected direct-to-LDS variants and the
    // non-square bf16 tiles, whole tiles and wide access, carry it
    const EpiFns* ef = nullptr;
    if (c.epi) {
        if (!aligned) return GEMM_ERR_NOT_SUPPORTED;
        ef = epi_fns_for(id, op_dtype, out_bf16);
        if (!ef) return GEMM_ERR_NOT_SUPPORTED;
    }
    pl.id = id;
    pl.sk = sk;
    pl.aligned = aligned;
    pl.nn_t = nn_t;
    pl.sk_fn = sk > 0 ? sk_launchers(vr, op_dtype, out_bf16, c.epi) : nullptr;
    pl.ef = ef;
    return GEMM_OK;
}

}  // namespace
}  // namespace dg

extern "C" {

gemm_status_t gemm_create(gemm_handle_t* out)
{
    if (!out) return GEMM_ERR_INVALID_VALUE;
    // a variable that is set, non-empty and not "0" turns its switch on
    auto env_on = [](const char* name) {
        const char* v = std::getenv(name);
        return v && v[0] != '\0' && std::strcmp(v, "0") != 0 ? 1 : 0;
    };
    gemm_handle_t h = new (std::nothrow) gemm_handle_s{
        -1, -1, -1, 0, nullptr, 0, dg::SK_SPIN_DEFAULT, env_on("GEMM_LOG"),
        env_on("GEMM_DEBUG_FAIL_LAUNCH"), 0, 0, {}};
    if (!h) return GEMM_ERR_ALLOC;
    *out = h;
    return GEMM_OK;
}

gemm_status_t gemm_destroy(gemm_handle_t h)
{
    delete h;
    return GEMM_OK;
}

const char* gemm_status_string(gemm_status_t s)
{
    switch (s) {
    case GEMM_OK: return "GEMM_OK";
    case GEMM_ERR_INVALID_VALUE: return "GEMM_ERR_INVALID_VALUE";
    case GEMM_ERR_NOT_SUPPORTED: return "GEMM_ERR_NOT_SUPPORTED";
    case GEMM_ERR_HIP: return "GEMM_ERR_HIP";
    case GEMM_ERR_ALLOC: return "GEMM_ERR_ALLOC";
    case GEMM_ERR_STREAM_K: return "GEMM_ERR_STREAM_K";
    }
    return "unknown status";
}

int gemm_variant_count(void) { return (int)dg::table().size(); }

const char* gemm_variant_name(int id)
{
    if (id < 0 || id >= gemm_variant_count()) return nullptr;
    return dg::table()[id].name;
}

int gemm_variant_dtype(int id)
{
    if (id < 0 || id >= gemm_variant_count()) return -1;
    return dg::table()[id].dtype;
}

gemm_status_t gemm_variant_tile(int id, int* bm, int* bn, int* bk)
{
    if (id < 0 || id >= gemm_variant_count()) return GEMM_ERR_INVALID_VALUE;
    const dg::Variant& v = dg::table()[id];
    if (bm) *bm = v.bm;
    if (bn) *bn = v.bn;
    if (bk) *bk = v.bk;
    return GEMM_OK;
}

gemm_status_t gemm_variant_pipeline(int id, int* stages, int* ahead)
{
    if (id < 0 || id >= gemm_variant_count()) return GEMM_ERR_INVALID_VALUE;
    const dg::Variant& v = dg::table()[id];
    if (stages) *stages = v.stages;
    if (ahead) *ahead = v.ahead;
    return GEMM_OK;
}

gemm_status_t gemm_set_planning_model(int cus, const int* occupancy, int count)
{
    if (cus < 0 || (occupancy && count != gemm_variant_count()) || count > dg::MAX_VARIANTS ||
        count < 0)
        return GEMM_ERR_INVALID_VALUE;
    if (occupancy)
        for (int i = 0; i < count; ++i)
            if (occupancy[i] < 0) return GEMM_ERR_INVALID_VALUE;
    for (int i = 0; i < dg::MAX_VARIANTS; ++i)
        dg::g_model_occ[i].store(occupancy && i < count ? occupancy[i] : 0,
                                 std::memory_order_relaxed);
    dg::g_model_cus.store(cus, std::memory_order_relaxed);
    return GEMM_OK;
}

int gemm_variant_occupancy(int id)
{
    if (id < 0 || id >= gemm_variant_count()) return -1;
    const int n = dg::table()[id].occ();
    return n > 0 ? n : -1;
}

gemm_status_t gemm_set_variant(gemm_handle_t h, int id)
{
    if (!h || id < -1 || id >= gemm_variant_count()) return GEMM_ERR_INVALID_VALUE;
    h->forced_variant = id;
    return GEMM_OK;
}

int gemm_last_variant(gemm_handle_t h) { return h ? h->last_variant : -1; }

int gemm_last_stream_k(gemm_handle_t h) { return h ? h->last_stream_k : -1; }

gemm_status_t gemm_set_stream_k_poll_limit(gemm_handle_t h, int polls)
{
    if (!h || polls < -1) return GEMM_ERR_INVALID_VALUE;
    h->sk_spin = polls < 0 ? dg::SK_SPIN_DEFAULT : polls;
    return GEMM_OK;
}

gemm_status_t gemm_stream_k_status(gemm_handle_t h, hipStream_t stream)
{
    using namespace dg;
    if (!h) return GEMM_ERR_INVALID_VALUE;
    gemm_status_t st = GEMM_OK;
    if (h->ws) st = check_and_clear(h->ws, stream);
    // the current device's gemm_run_no_alloc scratch, once it is set up
    const int dev = current_device();
    void* sp = dev >= 0 && dev < MAX_DEVICES ? scratch_addr[dev].load(std::memory_order_acquire)
                                             : nullptr;
    if (sp && st != GEMM_ERR_HIP) {
        const gemm_status_t s2 = check_and_clear(sp, stream);
        if (s2 != GEMM_OK) st = s2;
    }
    return st;
}

size_t gemm_stream_k_workspace_bytes(void)
{
    using namespace dg;
    size_t most = 0;
    for (const Variant& v : table()) {
        if (!v.sk_occ) continue;
        const size_t g = std::min<size_t>((size_t)device_cus() * variant_occupancy(v), SK_MAX_WG);
        most = std::max(most, g * v.bm * v.bn * sizeof(float));
    }
    return SK_FLAG_BYTES + most;
}

gemm_status_t gemm_set_workspace(gemm_handle_t h, void* ws, size_t bytes, hipStream_t stream)
{
    using namespace dg;
    if (!h) return GEMM_ERR_INVALID_VALUE;
    if (!ws || bytes == 0) {
        h->ws = nullptr;
        h->ws_bytes = 0;
        return GEMM_OK;
    }
    if (!aligned_to(ws, 256) || bytes < SK_FLAG_BYTES) return GEMM_ERR_INVALID_VALUE;
    unsigned* flags = static_cast<unsigned*>(ws);
    int n = SK_FLAG_WORDS;
    void* kargs[] = {&flags, &n};
    if (hipLaunchKernel(reinterpret_cast<const void*>(&clear_flags_kernel), dim3(16), dim3(256),
                        kargs, 0, stream) != hipSuccess)
        return GEMM_ERR_HIP;
    h->ws = ws;
    h->ws_bytes = bytes;
    return GEMM_OK;
}

gemm_status_t gemm_set_stream_k(gemm_handle_t h, int mode)
{
    if (!h || mode < -1 || mode > 1) return GEMM_ERR_INVALID_VALUE;
    h->stream_k_mode = mode;
    return GEMM_OK;
}

int gemm_select_variant(gemm_dtype_t dtype, gemm_op_t transA, gemm_op_t transB, int64_t M,
                        int64_t N, int64_t K)
{
    if ((dtype != GEMM_DTYPE_F32 && dtype != GEMM_DTYPE_BF16_F32 && dtype != GEMM_DTYPE_BF16_BF16) ||
        (transA != GEMM_OP_N && transA != GEMM_OP_T) || (transB != GEMM_OP_N && transB != GEMM_OP_T))
        return -1;
    if (M < 0 || N < 0 || K < 0) return -1;
    // a call with element-aligned, tightly packed operands, no workspace and
    // no fused epilogue
    dg::CallDesc cd;
    cd.dtype = dtype;
    cd.a_kc = transA == GEMM_OP_N;
    cd.b_kc = transB == GEMM_OP_T;
    cd.M = M;
    cd.N = N;
    cd.K = K;
    cd.lda = std::max<int64_t>(1, cd.a_kc ? K : M);
    cd.ldb = std::max<int64_t>(1, cd.b_kc ? K : N);
    cd.epi = false;
    cd.wide = true;
    cd.rows16 = (cd.lda * (dtype == GEMM_DTYPE_F32 ? 4 : 2)) % 16 == 0 &&
                (cd.ldb * (dtype == GEMM_DTYPE_F32 ? 4 : 2)) % 16 == 0;
    cd.forced = -1;
    cd.sk_mode = -1;
    cd.ws_bytes = 0;
    dg::Plan pl;
    return dg::plan_call(cd, pl) == GEMM_OK ? pl.id : -1;
}

static gemm_status_t run_gemm(gemm_handle_t h, gemm_op_t transA, gemm_op_t transB, int64_t M,
                              int64_t N, int64_t K, float alpha, const void* A, int64_t lda,
                              const void* B, int64_t ldb, float beta, const void* C, int64_t ldc,
                              void* D, int64_t ldd, gemm_dtype_t dtype, const gemm_epilogue_t* ep,
                              void* ws, size_t ws_bytes, hipStream_t stream)
{
    using namespace dg;
    if (!h) return GEMM_ERR_INVALID_VALUE;
    if ((transA != GEMM_OP_N && transA != GEMM_OP_T) || (transB != GEMM_OP_N && transB != GEMM_OP_T))
        return GEMM_ERR_INVALID_VALUE;
    if (dtype != GEMM_DTYPE_F32 && dtype != GEMM_DTYPE_BF16_F32 && dtype != GEMM_DTYPE_BF16_BF16)
        return GEMM_ERR_INVALID_VALUE;
    if (M < 0 || N < 0 || K < 0) return GEMM_ERR_INVALID_VALUE;
    if (ep) {
        if (ep->activation != GEMM_ACT_NONE && ep->activation != GEMM_ACT_RELU &&
            ep->activation != GEMM_ACT_GELU)
            return GEMM_ERR_INVALID_VALUE;
        if (ep->clamp && !(ep->clamp_lo <= ep->clamp_hi)) return GEMM_ERR_INVALID_VALUE;  // NaN too
    }
    // a fused epilogue with something to do (bias, activation or clamp)
    const bool epi = ep && (ep->bias || ep->activation != GEMM_ACT_NONE || ep->clamp);
    const bool out_bf16 = dtype == GEMM_DTYPE_BF16_BF16;
    const int64_t es_out = out_bf16 ? 2 : 4;  // bytes per element of C and D
    const int64_t one = 1;
    const int64_t min_lda = transA == GEMM_OP_N ? std::max(one, K) : std::max(one, M);
    const int64_t min_ldb = transB == GEMM_OP_N ? std::max(one, N) : std::max(one, K);
    const int64_t min_ldcd = std::max(one, N);
    if (lda < min_lda || ldb < min_ldb || ldd < min_ldcd) return GEMM_ERR_INVALID_VALUE;
    if (beta != 0.0f && ldc < min_ldcd) return GEMM_ERR_INVALID_VALUE;
    h->last_variant = -1;
    h->last_stream_k = 0;
    if (M == 0 || N == 0) return GEMM_OK;
    const bool reads_ab = K > 0 && alpha != 0.0f;
    if (!D) return GEMM_ERR_INVALID_VALUE;
    if (beta != 0.0f && !C) return GEMM_ERR_INVALID_VALUE;
    if (reads_ab && (!A || !B)) return GEMM_ERR_INVALID_VALUE;
    if (M > INT_MAX || N > INT_MAX || K > INT_MAX || lda > INT_MAX || ldb > INT_MAX ||
        ldd > INT_MAX || (beta != 0.0f && ldc > INT_MAX))
        return GEMM_ERR_NOT_SUPPORTED;
    const int64_t span_d = ((M - 1) * ldd + N) * es_out;
    if (beta != 0.0f) {
        const int64_t span_c = ((M - 1) * ldc + N) * es_out;
        if (static_cast<const void*>(C) == static_cast<const void*>(D)) {
            if (ldc != ldd) return GEMM_ERR_INVALID_VALUE;
        } else if (ranges_overlap(C, span_c, D, span_d)) {
            return GEMM_ERR_INVALID_VALUE;
        }
    }
    if (epi && ep->bias) {
        // the bias is read while D is written: it must lie outside D
        if (ranges_overlap(ep->bias, N * es_out, D, span_d)) return GEMM_ERR_INVALID_VALUE;
        if (!aligned_to(ep->bias, es_out)) return GEMM_ERR_NOT_SUPPORTED;
    }

    GemmArgs a;
    a.A = A;
    a.B = B;
    a.C = beta != 0.0f ? static_cast<const float*>(C) : nullptr;  // element type per dtype
    a.D = static_cast<float*>(D);
    a.lda = lda;
    a.ldb = ldb;
    a.ldc = beta != 0.0f ? ldc : 0;
    a.ldd = ldd;
    a.M = (int)M;
    a.N = (int)N;
    a.K = (int)K;
    a.alpha = alpha;
    a.beta = beta;
    // 16-byte accesses need only element alignment: the memory system serves
    // unaligned vector loads and stores whole
    a.c_vec = beta != 0.0f && aligned_to(C, es_out);
    a.d_vec = aligned_to(D, es_out);
    a.sk_partials = nullptr;
    a.sk_flags = nullptr;
    a.sk_error = nullptr;
    a.sk_spin = h->sk_spin;
    a.bias = epi ? ep->bias : nullptr;
    a.act = epi ? (int)ep->activation : EPI_ACT_NONE;
    a.clamp = epi && ep->clamp;
    a.clamp_lo = a.clamp ? ep->clamp_lo : 0.0f;
    a.clamp_hi = a.clamp ? ep->clamp_hi : 0.0f;

    if (!reads_ab) {
        if (h->fail_launch) return GEMM_ERR_HIP;
        const int64_t blocks = std::min<int64_t>(ceil_div(M * N, 256), 65536);
        void* args[] = {&a};
        const void* k = out_bf16 ? reinterpret_cast<const void*>(&scale_c_kernel<bf16_t>)
                                 : reinterpret_cast<const void*>(&scale_c_kernel<float>);
        hipError_t e = hipLaunchKernel(k, dim3((unsigned)blocks), dim3(256), args, 0, stream);
        return e == hipSuccess ? GEMM_OK : GEMM_ERR_HIP;
    }

    CallDesc cd;
    cd.dtype = dtype;
    cd.a_kc = transA == GEMM_OP_N;
    cd.b_kc = transB == GEMM_OP_T;
    cd.M = M;
    cd.N = N;
    cd.K = K;
    cd.lda = lda;
    cd.ldb = ldb;
    cd.epi = epi;
    // wide (16-byte) operand access needs element-aligned A and B only
    const int64_t es = dtype == GEMM_DTYPE_F32 ? 4 : 2;
    cd.wide = aligned_to(A, es) && aligned_to(B, es);
    cd.rows16 = aligned_to(A, 16) && aligned_to(B, 16) && (lda * es) % 16 == 0 &&
                (ldb * es) % 16 == 0;
    cd.forced = h->forced_variant;
    cd.sk_mode = h->stream_k_mode;
    cd.ws_bytes = ws ? ws_bytes : 0;
    Plan pl;
    const gemm_status_t ps = plan_call(cd, pl);
    if (ps != GEMM_OK) return ps;
    const int id = pl.id, sk = pl.sk;
    const bool aligned = pl.aligned, nn_t = pl.nn_t, a_kc = cd.a_kc, b_kc = cd.b_kc;
    const Variant& vr = table()[id];
    a.tiles_m = (int)ceil_div(M, vr.bm);
    a.tiles_n = (int)ceil_div(N, vr.bn);
    // 4 tile-rows per group measured best on 8192^3 bf16 (groups of 1, 2, 3, 4, 6,
    // 8, 16 and 32 tried, with and without the XCD renumbering)
    a.group_m = std::min(a.tiles_m, 4);
    // whole tiles: the transposed-output launch tiles N by BM and M by BN
    const int64_t grid = nn_t ? ceil_div(N, vr.bm) * ceil_div(M, vr.bn)
                              : (int64_t)a.tiles_m * a.tiles_n;
    if (grid > INT_MAX) return GEMM_ERR_NOT_SUPPORTED;
    if (h->fail_launch) return GEMM_ERR_HIP;
    hipError_t e;
    const EpiFns* ef = pl.ef;
    if (sk > 0) {
        // the plan only takes grids whose slots fit in the workspace
        const size_t need = SK_FLAG_BYTES + (size_t)sk * vr.bm * vr.bn * sizeof(float);
        if (need > cd.ws_bytes) return GEMM_ERR_NOT_SUPPORTED;
        a.sk_flags = static_cast<unsigned*>(ws);
        a.sk_error = a.sk_flags + SK_MAX_WG;
        a.sk_partials = reinterpret_cast<float*>(static_cast<char*>(ws) + SK_FLAG_BYTES);
        e = pl.sk_fn[a_kc][b_kc](a, sk, stream);
    } else if (nn_t) {
        GemmArgs t = a;
        t.A = B;
        t.B = A;
        t.lda = ldb;
        t.ldb = lda;
        t.M = (int)N;
        t.N = (int)M;
        t.tiles_m = (int)ceil_div(N, vr.bm);
        t.tiles_n = (int)ceil_div(M, vr.bn);
        t.group_m = std::min(t.tiles_m, 4);
        e = (ef ? ef->nn_t : out_bf16 ? vr.bo_nn_t_fn : vr.nn_t_fn)(t, (int)grid, stream);
    } else if (ef) {
        e = ef->fn[a_kc][b_kc](a, (int)grid, stream);
    } else {
        e = (out_bf16 ? vr.bo_fn : vr.fn)[aligned][a_kc][b_kc](a, (int)grid, stream);
    }
    if (e != hipSuccess) return GEMM_ERR_HIP;
    h->last_variant = id;
    h->last_stream_k = sk;
    if (h->log) {
        static const char* const dt_name[3] = {"f32", "bf16_f32", "bf16_bf16"};
        std::fprintf(stderr,
                     "gemm: %s %c%c M=%lld N=%lld K=%lld dtype=%s grid=%lld stream_k=%d "
                     "as_transpose=%d epilogue=%d\n",
                     vr.name, transA == GEMM_OP_N ? 'N' : 'T', transB == GEMM_OP_N ? 'N' : 'T',
                     (long long)M, (long long)N, (long long)K, dt_name[dtype],
                     (long long)(sk > 0 ? sk : grid), sk, nn_t ? 1 : 0, epi ? 1 : 0);
    }
    return GEMM_OK;
}

gemm_status_t gemm_run(gemm_handle_t h, gemm_op_t transA, gemm_op_t transB, int64_t M, int64_t N,
                       int64_t K, float alpha, const void* A, int64_t lda, const void* B, int64_t ldb,
                       float beta, const void* C, int64_t ldc, void* D, int64_t ldd,
                       gemm_dtype_t dtype, hipStream_t stream)
{
    if (!h) return GEMM_ERR_INVALID_VALUE;
    return run_gemm(h, transA, transB, M, N, K, alpha, A, lda, B, ldb, beta, C, ldc, D, ldd, dtype,
                    nullptr, h->ws, h->ws_bytes, stream);
}

gemm_status_t gemm_run_no_alloc(gemm_handle_t h, gemm_op_t transA, gemm_op_t transB, int64_t M,
                                int64_t N, int64_t K, float alpha, const void* A, int64_t lda,
                                const void* B, int64_t ldb, float beta, const void* C,
                                int64_t ldc, void* D, int64_t ldd, gemm_dtype_t dtype,
                                hipStream_t stream)
{
    using namespace dg;
    if (!h) return GEMM_ERR_INVALID_VALUE;
    // set up (first call on this device) only once the arguments look like a
    // call that launches something; run_gemm validates them all again
    void* ws = nullptr;
    if (M > 0 && N > 0 && D) {
        ws = scratch_address(stream);
        if (!ws) return GEMM_ERR_HIP;
    }
    return run_gemm(h, transA, transB, M, N, K, alpha, A, lda, B, ldb, beta, C, ldc, D, ldd, dtype,
                    nullptr, ws, GEMM_NO_ALLOC_SCRATCH_BYTES, stream);
}

gemm_status_t gemm_run_epilogue(gemm_handle_t h, gemm_op_t transA, gemm_op_t transB, int64_t M,
                                int64_t N, int64_t K, float alpha, const void* A, int64_t lda,
                                const void* B, int64_t ldb, float beta, const void* C,
                                int64_t ldc, void* D, int64_t ldd, gemm_dtype_t dtype,
                                const gemm_epilogue_t* epilogue, hipStream_t stream)
{
    if (!h) return GEMM_ERR_INVALID_VALUE;
    return run_gemm(h, transA, transB, M, N, K, alpha, A, lda, B, ldb, beta, C, ldc, D, ldd, dtype,
                    epilogue, h->ws, h->ws_bytes, stream);
}

}  // extern "C"
