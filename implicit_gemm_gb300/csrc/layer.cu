// Layers of the C ABI (declared in include/wgrad.h): the matrix product with bias,
// activation, dropout and residual, its gradients, the same by expert, and the
// activation alone.  Validation, plans, workspace layout and launches; no device
// memory is allocated here.
#include <cuda.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stddef.h>
#include <stdio.h>

#include <algorithm>
#include <string>

#include "../../include/wgrad.h"
#include "host.h"
#include "k_linear.cuh"

namespace wg {

cudaError_t read_layer_status(unsigned int* v) { return cudaMemcpyFromSymbol(v, g_status, sizeof *v); }
cudaError_t write_layer_status(unsigned int v) { return cudaMemcpyToSymbol(g_status, &v, sizeof v); }

}  // namespace wg

namespace {

using wg::aligned16;
using wg::cuda_fail;
using wg::num_sms;
using wg::set_err;

// Elements that a layout may span: their bytes and the sums of their addresses stay in 64 bits.
constexpr long long kMaxSpan = 1LL << 48;
constexpr long long kMaxTokens = (1LL << 31) - 65536;
constexpr int kMaxFeatures = 1 << 20;

int esize(int dtype) { return dtype == WG_FP32 ? 4 : 2; }
bool dtype_ok(int d) { return d == WG_FP32 || d == WG_BF16 || d == WG_FP16; }
bool act_ok(int a) { return a >= WG_ACT_NONE && a <= WG_ACT_SILU; }
bool aligned_to(const void* p, int bytes) { return (reinterpret_cast<uintptr_t>(p) & (uintptr_t)(bytes - 1)) == 0; }
size_t up256(size_t n) { return (n + 255) / 256 * 256; }

// What a call reads or writes: rows of `cols` elements of `es` bytes, `ld` apart, `count` matrices `stride` apart.
struct Tensor {
    const char* name;
    const void* p;
    long long rows, cols, ld;
    int es;
    long long count, stride;
    long long bytes() const
    {
        if (!p || rows <= 0 || count <= 0) return 0;
        return ((count - 1) * stride + (rows - 1) * ld + cols) * es;
    }
};

// Whether two tensors whose rows are one stride apart lie side by side in it, as columns of one buffer do.
bool side_by_side(const Tensor& a, const Tensor& b)
{
    const Tensor& r = a.rows > 1 ? a : b;
    const long long row = r.ld * r.es;
    for (const Tensor* t : {&a, &b})
        if ((t->rows > 1 && t->ld * t->es != row) || (t->count > 1 && t->stride * t->es % row)) return false;
    const uintptr_t x = reinterpret_cast<uintptr_t>(a.p), y = reinterpret_cast<uintptr_t>(b.p);
    const long long d = y >= x ? (long long)((y - x) % (uintptr_t)row) : (row - (long long)((x - y) % (uintptr_t)row)) % row;
    return d >= a.cols * a.es && d + b.cols * b.es <= row;
}

// The first `outputs` of n tensors are written: none of them may share bytes with another one, but for pairs that
// are the same elements (same address, type and strides) where `same` allows it.
int check_tensors(const Tensor* t, int n, int outputs, int same_a, int same_b, int same_c = -1)
{
    for (int i = 0; i < n; ++i)
        if (!aligned_to(t[i].p, t[i].es)) return set_err(WG_ERR_MISALIGNED, std::string(t[i].name) + " is not aligned to its elements");
    for (int i = 0; i < outputs; ++i)
        for (int j = 0; j < n; ++j) {
            if (i == j) continue;
            const Tensor &a = t[i], &b = t[j];
            const long long na = a.bytes(), nb = b.bytes();
            const uintptr_t x = reinterpret_cast<uintptr_t>(a.p), y = reinterpret_cast<uintptr_t>(b.p);
            if (!na || !nb || x >= y + (uintptr_t)nb || y >= x + (uintptr_t)na || side_by_side(a, b)) continue;
            const bool equal = x == y && a.es == b.es && a.ld == b.ld && a.rows == b.rows && a.cols == b.cols;
            if (i == same_a && (j == same_b || j == same_c) && equal) continue;
            return set_err(WG_ERR_INVALID_ARGUMENT, std::string(a.name) + " overlaps " + b.name);
        }
    return WG_OK;
}

int check_workspace(size_t need, const void* workspace, size_t ws_bytes)
{
    if (need == 0) return WG_OK;
    if (!workspace || ws_bytes < need) {
        char buf[160];
        snprintf(buf, sizeof buf, "workspace of %zu bytes needed (got %zu%s)", need, ws_bytes, workspace ? "" : ", NULL");
        return set_err(WG_ERR_WORKSPACE, buf);
    }
    if (!aligned16(workspace)) return set_err(WG_ERR_MISALIGNED, "workspace must be 16-byte aligned");
    return WG_OK;
}

template <typename... P, typename... A>
int launch(const char* what, void (*k)(P...), dim3 grid, dim3 block, cudaStream_t stream, A... args)
{
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    unsigned na = 0;
    wg::pdl_config(&cfg, attr, &na, stream);
    cfg.gridDim = grid;
    cfg.blockDim = block;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, k, args...);
    return e == cudaSuccess ? WG_OK : cuda_fail(what, e);
}

// Dropout of probability p in [0, 1) on the grid of 2^-16.
void set_dropout(wg::LayerTail* t, float p, unsigned long long seed, unsigned long long offset, const unsigned long long* counter)
{
    const unsigned thr = (unsigned)std::min(65535.0, floor(65536.0 * (double)p + 0.5));
    t->thr = thr << 16;
    t->gain = (float)(65536.0 / (65536.0 - thr));
    for (unsigned i = 0; i < 10; ++i)
        t->key[i] = make_uint2((unsigned)seed + i * 0x9E3779B9u, (unsigned)(seed >> 32) + i * 0xBB67AE85u);
    t->offset = offset, t->counter = counter;
}

int check_factors(int act, float dropout, const unsigned long long* counter)
{
    if (!act_ok(act)) return set_err(WG_ERR_INVALID_ARGUMENT, "activation must be one of wg_activation_kind");
    if (!(dropout >= 0.f && dropout < 1.f)) return set_err(WG_ERR_INVALID_ARGUMENT, "dropout must be in [0, 1)");
    if (!aligned_to(counter, 8)) return set_err(WG_ERR_MISALIGNED, "counter must be 8-byte aligned");
    return WG_OK;
}

// 16-byte accesses of eight elements: every row's eight-column chunks lie on 16 bytes.
bool vec_rows(const void* p, long long ld, int cols, int es, long long stride = 0)
{
    return cols % 8 == 0 && (ld * es) % 16 == 0 && (stride * es) % 16 == 0 && aligned16(p);
}

// 4-byte accesses of two 16-bit elements.
bool pair_rows(const void* p, long long ld, int cols, int es, long long stride = 0)
{
    return es == 2 && cols % 2 == 0 && ld % 2 == 0 && stride % 2 == 0 && aligned_to(p, 4);
}

int log2_floor(long long n)
{
    int b = 0;
    while ((2LL << b) <= n) ++b;
    return b;
}

// dbias of `experts` from `chunks` partial sums in all; as many threads a column as leave each some four.
void plan_join(wg::SumParams* m, int experts, long long chunks, int threads)
{
    m->ny_log = std::min(5, log2_floor(std::max(1LL, chunks / experts / 4)));
    const int nx = threads >> m->ny_log;
    m->across = (m->dim + nx - 1) / nx, m->units = m->across * experts;
}
int join_columns(wg::SumParams m, int experts, long long chunks, cudaStream_t s)
{
    plan_join(&m, experts, chunks, wg::kJoinThreads);
    return launch("column_join_kernel launch", wg::column_join_kernel, dim3((unsigned)m.across, (unsigned)experts), dim3(wg::kJoinThreads), s, m);
}

// ---------------------------------------------------------------- products
struct LinPlan {
    wg_linear_problem p;
    wg_linear_call call;
    int M, N, kb;             // columns of the result, rows (weight gradient), 64-wide blocks of the sum
    int bt, split, stages, stage_bytes, pairs;
    bool few;                 // linear_rows_kernel
    long long chunks;         // of the longest sum (a part's, or an expert's that has every row)
    bool pack_a, pack_b;      // operands that TMA cannot read
    long long part_rows, ldp;
    int sum_rows;             // rows of a partial sum of dbias
    long long sum_chunks;
    size_t off_a, off_b, off_part, off_sum, off_first, bytes;
};

// Blocks of 64 per sum in tensor memory.  Truncation takes up to 0.95e-7 n of a sum of n
// MMAs (16 terms each) of equal signs, a few times less of mixed ones: 6e-6 of an fp32
// result's (n = 64), 2e-4 of a 16-bit one's (n = 2048), 0.4 of fp16's rounding.
constexpr int kChunkFp32 = 16, kChunk16 = 512;
int lin_chunk(const wg_linear_problem& q) { return q.out_dtype == WG_FP32 ? kChunkFp32 : kChunk16; }

// Rows up to which the weight gradient's product makes dbias itself (512 x 1024 to 1000 6.8 us against 12.7 with a
// kernel before it, 2048 x 2560 to 4096 38.8 against 45.6; 4000 x 128 to 300 30 against 19).
constexpr int kFewSums = 2048;

// Rows up to which the forward product is linear_rows_kernel's: eight at a time; 16 of one
// weight matrix below 64 MB (4096 x 4096 for 9 rows 9.7 us against 14.1 on the tensor-core tiles,
// 4096 x 16384 for 16 rows 31 against 25), and 16 of experts.  Where the tiles
// would need a copy of the weights, 16 of any matrix (12 rows of 8191 x 7168 61 against 75, of 8190 x 8192 39
// against 84) and 64 of experts with eight each at most on average, which are not known here (20 rows of 4 experts'
// 3918 x 3840, 5 each, 40 against 80; 64 of 16 experts' 2047 x 2048, 4 each, 49 against 78; of 8 experts' 26 against
// 45, but if one expert has them all 24 against 18).
constexpr int kFewRows = 16, kFewCopied = wg::kRowsMost;
bool few_rows(const wg_linear_problem& q)
{
    const bool copied = q.ld_in % 8 || q.ld_weight % 8 || (q.experts > 1 && q.weight_stride % 8);
    return q.tokens <= 8 || (q.tokens <= kFewRows && (q.experts > 1 || (long long)q.in * q.out < (32LL << 20) || copied)) ||
           (copied && q.tokens <= std::min(kFewCopied, 8 * q.experts));
}

// us of a block of 64 of a tile's sum on every pair at once, by the tile's MMA columns
// (measured on the update's products: 0.33 for 256, 0.27 for 128, L2 to shared memory being
// what bounds the narrower ones).
double block_us(int wide) { return 0.21 + 0.12 * wide / 256; }

int lin_plan(const wg_linear_problem* p, int call, LinPlan* pl)
{
    if (!p) return set_err(WG_ERR_INVALID_ARGUMENT, "problem is NULL");
    if (call < WG_LINEAR_FORWARD || call > WG_LINEAR_BWD_WEIGHT) return set_err(WG_ERR_INVALID_ARGUMENT, "call must be one of wg_linear_call");
    if (p->tokens < 0 || p->in < 1 || p->out < 1 || p->experts < 0)
        return set_err(WG_ERR_INVALID_ARGUMENT, "tokens and experts must be at least 0, in and out at least 1");
    if (p->tokens > kMaxTokens || p->in > kMaxFeatures || p->out > kMaxFeatures || p->experts > wg::kLinMaxExperts)
        return set_err(WG_ERR_NOT_SUPPORTED, "tokens up to 2^31-65536, in and out up to 2^20 and experts up to 1024 are supported");
    if (p->in_dtype != WG_BF16 && p->in_dtype != WG_FP16) return set_err(WG_ERR_INVALID_ARGUMENT, "in_dtype must be WG_BF16 or WG_FP16");
    if (!dtype_ok(p->out_dtype) || !dtype_ok(p->bias_dtype))
        return set_err(WG_ERR_INVALID_ARGUMENT, "out_dtype and bias_dtype must be WG_FP32, WG_BF16 or WG_FP16");
    if (p->offset_bits != 32 && p->offset_bits != 64) return set_err(WG_ERR_INVALID_ARGUMENT, "offset_bits must be 32 or 64");
    const int st = check_factors(p->activation, p->dropout, p->counter);
    if (st) return st;
    *pl = LinPlan();
    pl->p = *p, pl->call = (wg_linear_call)call;
    wg_linear_problem& q = pl->p;
    const bool weight = call == WG_LINEAR_BWD_WEIGHT, data = call == WG_LINEAR_BWD_DATA;
    const int ycols = data ? q.in : q.out;
    if (q.ld_in == 0) q.ld_in = q.in;
    if (q.ld_out == 0) q.ld_out = q.out;
    if (q.ld_weight == 0) q.ld_weight = q.in;
    if (q.ld_z == 0) q.ld_z = ycols;
    if (q.ld_residual == 0) q.ld_residual = ycols;
    if (q.ld_in < q.in || q.ld_out < q.out || q.ld_weight < q.in || q.ld_z < ycols || q.ld_residual < ycols)
        return set_err(WG_ERR_INVALID_ARGUMENT, "a row stride must be 0 or at least the row's columns");
    const long long n = std::max(q.tokens, 1LL), far = kMaxSpan / n;
    if (q.ld_in > far || q.ld_out > far || q.ld_z > far || q.ld_residual > far || q.ld_weight > kMaxSpan / q.out)
        return set_err(WG_ERR_INVALID_ARGUMENT, "a row stride is larger than any memory");
    const int ne = std::max(q.experts, 1);
    if (q.weight_stride == 0 || ne == 1) q.weight_stride = q.out * q.ld_weight;
    if (q.weight_stride < (q.out - 1) * q.ld_weight + q.in)
        return set_err(WG_ERR_INVALID_ARGUMENT, "weight_stride makes experts' matrices overlap");
    if (q.weight_stride > kMaxSpan / ne) return set_err(WG_ERR_INVALID_ARGUMENT, "weight_stride is larger than any memory");

    // Few rows: the forward product that reads the weights once, in one launch.
    if (call == WG_LINEAR_FORWARD && few_rows(q)) {
        pl->few = true;
        pl->bytes = 256;
        return WG_OK;
    }
    pl->M = call == WG_LINEAR_FORWARD ? q.out : q.in;
    pl->N = weight ? q.out : 0;
    pl->kb = ((weight ? (int)std::min<long long>((q.tokens + ne - 1) / ne, 1 << 30) : data ? q.out : q.in) + 63) / 64;
    pl->pairs = std::max(1, num_sms() / 2);
    const long long im = (pl->M + 255) / 256, rows = weight ? q.out : q.tokens;
    if (im * (weight ? (long long)ne * ((q.out + 31) / 32) : (q.tokens + 31) / 32 + ne) > 0x7fffffffLL)
        return set_err(WG_ERR_NOT_SUPPORTED, "more tiles than one launch covers");
    // Rows of a tile and parts of the sum, by the time of the pair with most of them: its
    // blocks, an epilogue, and what parts cost (a kernel that joins them, and their fp32
    // sums written and read).  Experts' rows are taken as even: each leaves half a tile
    // unused on average.
    const long long used = weight ? ne : std::min<long long>(ne, n);
    pl->ldp = (pl->M + 7) / 8 * 8;
    pl->part_rows = weight ? (long long)ne * q.out : q.tokens;
    // us of what follows the products of a tile of 256 x 256, measured with short sums: its stores (2.0
    // in 16 bits, 3 in 32), an activation 2, dropout 4; twice that in the kernel for long sums of fp32 results.
    double tail256 = q.out_dtype == WG_FP32 ? 3.0 : 2.0;
    if (!weight) tail256 += (q.activation != WG_ACT_NONE ? 2.0 : 0.0) + (q.dropout > 0.f ? 4.0 : 0.0);
    if (q.out_dtype == WG_FP32 && pl->kb > kChunkFp32) tail256 *= 2.0;
    double best = 1e30;
    for (int bt = 256; bt >= 32; bt -= 32) {
        const int least = (int)std::min<long long>((rows + 31) / 32 * 32, 256);
        if (bt > std::max(least, 32)) continue;
        const long long along = weight ? ne * ((rows + bt - 1) / bt) : q.experts ? std::max(used, (2 * rows + bt * used) / (2 * bt)) : (rows + bt - 1) / bt;
        const long long tiles = std::max(1LL, im * along);
        for (int s = 1; s <= 16; ++s) {
            if (s > 1 && (tiles * s > 2 * pl->pairs || pl->kb < 4 * s)) break;
            // A pair's tiles: the products of one beside what follows those of the tile before.
            const double rounds = (double)((tiles * s + pl->pairs - 1) / pl->pairs);
            const double main = ((pl->kb + s - 1) / s) * block_us(bt), tail = s > 1 ? 1.5 : 1.0 + (tail256 - 1.0) * bt / 256;
            double t = 3.0 + rounds * std::max(main, tail) + std::min(main, tail);
            if (s > 1) t += 3.0 + (double)s * pl->part_rows * pl->ldp * 8 / 1e7;
            if (t < best - 1e-9) best = t, pl->bt = bt, pl->split = s;
        }
    }
    const long long blocks = ((weight ? (q.tokens + 63) / 64 : pl->kb) + pl->split - 1) / pl->split;
    pl->chunks = (blocks + lin_chunk(q) - 1) / lin_chunk(q);
    pl->stage_bytes = wg::kLinABytes + (weight ? (pl->bt > 128 ? 16384 : 8192) : pl->bt * 64);
    pl->stages = std::min(wg::kLinMaxStages, wg::kLinRing / pl->stage_bytes);

    const auto direct = [](long long ld, long long stride) { return ld % 8 == 0 && stride % 8 == 0 && ld < (1LL << 38) && stride < (1LL << 38); };
    const long long wstride = ne > 1 ? q.weight_stride : 0;
    pl->pack_a = !(weight ? direct(q.ld_in, 0) : direct(q.ld_weight, wstride));
    pl->pack_b = !direct(weight || data ? q.ld_out : q.ld_in, 0);
    const auto packed = [](long long r, int cols) { return up256((size_t)r * ((cols + 7) / 8 * 8) * 2); };
    size_t o = 0;
    if (pl->pack_a) pl->off_a = o, o += weight ? packed(n, q.in) : packed((long long)ne * q.out, q.in);
    if (pl->pack_b) pl->off_b = o, o += packed(n, weight || data ? q.out : q.in);
    if (pl->split > 1) pl->off_part = o, o += up256((size_t)pl->split * pl->part_rows * pl->ldp * 4);
    if (weight) {
        // Rows of a partial sum: 64 for each of a block's eight rows of threads to have eight in
        // flight, more where that is still two blocks for every place on the GPU.
        const long long cols = (q.out + 255) / 256;
        pl->sum_rows = (int)std::max(64LL, std::min(512LL, q.tokens * cols / (12 * num_sms()) / 64 * 64));
        pl->sum_chunks = q.tokens / pl->sum_rows + ne + 1;
        pl->off_sum = o, o += up256((size_t)pl->sum_chunks * q.out * 4);
        pl->off_first = o, o += up256((size_t)(ne + 1) * 4);
    }
    pl->bytes = std::max<size_t>(o, 256);  // (callers need no case for a form without a workspace)
    return WG_OK;
}

// 16-bit matrices [batch][rows][cols], read in boxes of 64 columns by `box` rows.
int lin_map(CUtensorMap* tm, const void* base, int bf16, long long cols, long long rows, long long batch, long long ld, long long bs, int box)
{
    wg::EncodeTiledFn fn = wg::encode_fn();
    if (!fn) return set_err(WG_ERR_CUDA, "cuTensorMapEncodeTiled is not available from the driver");
    const cuuint64_t dims[3] = {(cuuint64_t)cols, (cuuint64_t)rows, (cuuint64_t)batch};
    // (One matrix: its stride is not used, and might be more than a map holds.)
    const cuuint64_t strides[2] = {(cuuint64_t)ld * 2, (cuuint64_t)(batch > 1 ? bs : ld) * 2};
    const cuuint32_t bx[3] = {64, (cuuint32_t)box, 1}, es[3] = {1, 1, 1};
    const CUresult r = fn(tm, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 3, const_cast<void*>(base), dims,
                          strides, bx, es, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                          CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    if (r != CUDA_SUCCESS) return set_err(WG_ERR_CUDA, "cuTensorMapEncodeTiled failed with CUresult " + std::to_string((int)r));
    return WG_OK;
}

// An operand of the products: 16-bit matrices that TMA reads as they are, or a copy of them in the workspace.
struct LinOperand {
    const void* p;
    long long rows;
    int cols;
    long long ld, batch, bs;
};
wg::PackParams lin_pack(LinOperand* o, char* to)
{
    const int per = (o->cols + 255) / 256, segments = (int)(o->rows * per);
    wg::PackParams k = {static_cast<const unsigned short*>(o->p), reinterpret_cast<unsigned short*>(to), o->rows, o->ld, o->bs,
                        (int)o->batch, o->cols, (o->cols + 7) / 8 * 8, segments, wg::fast_div((unsigned)per), wg::fast_div((unsigned)segments)};
    o->p = to, o->ld = k.ldp, o->bs = o->rows * k.ldp;
    return k;
}

// The chunked kernels' warps pass registers on (setmaxnreg), out of those that a launch takes: with fewer than
// they are written for, the epilogue's warps would wait for ever.  Asked of the built kernel, once.
template <int KIND>
int check_registers()
{
    static const int st = [] {
        cudaFuncAttributes a;
        const cudaError_t e = cudaFuncGetAttributes(&a, wg::linear_product_kernel<KIND, true>);
        return e != cudaSuccess ? -1 : a.numRegs;
    }();
    const int need = 128 * wg::kLinDirectRegs + 32 * wg::lin_epi_warps(true) * wg::kLinChunkedRegs;
    if (st * wg::lin_threads(true) >= need) return WG_OK;
    return set_err(WG_ERR_CUDA, "linear_product_kernel was built with " + std::to_string(st) + " registers a thread, fewer than it hands out");
}

// The kernels of a call, and what has to hold before they are launched.
struct LinKernels {
    void (*product)(CUtensorMap, CUtensorMap, wg::LinParams);
    void (*join)(wg::LinParams);
    int (*check)();
};
template <int KIND>
LinKernels lin_kernels(bool chunked)
{
    if (chunked) return {wg::linear_product_kernel<KIND, true>, wg::linear_join_kernel<KIND>, check_registers<KIND>};
    return {wg::linear_product_kernel<KIND, false>, wg::linear_join_kernel<KIND>, [] { return (int)WG_OK; }};
}

int product_launch(const LinPlan& pl, const LinKernels& k, const CUtensorMap& ma, const CUtensorMap& mb, const wg::LinParams& g, cudaStream_t s)
{
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[2];
    unsigned na = 0;
    attr[na].id = cudaLaunchAttributeClusterDimension;
    attr[na].val.clusterDim.x = 2;
    attr[na].val.clusterDim.y = attr[na].val.clusterDim.z = 1;
    ++na;
    wg::pdl_config(&cfg, attr, &na, s);
    cfg.gridDim = dim3((unsigned)(2 * g.pairs));
    cfg.blockDim = dim3(wg::lin_threads(pl.chunks > 1));
    cfg.dynamicSmemBytes = wg::kLinSmem;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, k.product, ma, mb, g);
    if (e != cudaSuccess) return cuda_fail("linear_product_kernel launch", e);
    if (pl.split == 1) return WG_OK;
    return launch("linear_join_kernel launch", k.join, dim3((unsigned)(g.join_blocks + (g.sums.part ? g.sums.units : 0))),
                  dim3(wg::kJoinBlock), s, g);
}

int columns_launch(const wg::ColumnParams& c, const LinPlan& pl, cudaStream_t s)
{
    const bool vec = vec_rows(c.dy, c.ld, c.N, 2);
    const int groups = (c.N + 7) / 8;
    const long long cols = (groups + (1 << c.cx_log) - 1) >> c.cx_log;
    const long long rows = std::min(pl.sum_chunks, (4LL * num_sms() + cols - 1) / cols);
    const auto kernel = vec ? wg::column_sum_kernel<wg::kActWide> : wg::column_sum_kernel<wg::kActShifted>;
    return launch("column_sum_kernel launch", kernel, dim3((unsigned)cols, (unsigned)std::max(1LL, rows)), dim3(256), s, c);
}

// w, or x of the weight gradient, is operand a (MMA rows); the other operand b.  dbias: few, sums that the product
// makes itself, or sums, partial sums made before it and what joins them.
int lin_run(const LinPlan& pl, const void* offsets, LinOperand a, LinOperand b, const wg::LayerTail& tail, char* ws, cudaStream_t s,
            const wg::FewSums* few = nullptr, const wg::ColumnParams* sums = nullptr, wg::SumParams* joined = nullptr)
{
    const wg_linear_problem& q = pl.p;
    if (!pl.pack_a && !aligned16(a.p)) return set_err(WG_ERR_MISALIGNED, "x, w or dy with 16-byte strides must be 16-byte aligned");
    if (!pl.pack_b && !aligned16(b.p)) return set_err(WG_ERR_MISALIGNED, "x, w or dy with 16-byte strides must be 16-byte aligned");
    wg::PackParams ka = {}, kb = {};
    if (q.tokens > 0) {
        if (pl.pack_a) ka = lin_pack(&a, ws + pl.off_a);
        if (pl.pack_b) kb = lin_pack(&b, ws + pl.off_b);
    } else {
        a.p = b.p = ws, a.ld = b.ld = 8LL * (kMaxFeatures / 8), a.rows = b.rows = 1, a.batch = 1, a.bs = a.ld;  // (never read)
    }
    // Whatever may fail comes before the first launch.
    const LinKernels kernels = pl.call == WG_LINEAR_FORWARD    ? lin_kernels<wg::kForward>(pl.chunks > 1)
                               : pl.call == WG_LINEAR_BWD_DATA ? lin_kernels<wg::kData>(pl.chunks > 1)
                                                               : lin_kernels<wg::kWeight>(pl.chunks > 1);
    const int bf16 = q.in_dtype == WG_BF16;
    CUtensorMap ma, mb;
    int st = lin_map(&ma, a.p, bf16, a.cols, a.rows, a.batch, a.ld, a.bs, pl.call == WG_LINEAR_FORWARD ? 128 : 64);
    if (!st) st = lin_map(&mb, b.p, bf16, b.cols, b.rows, 1, b.ld, 0, pl.call == WG_LINEAR_BWD_WEIGHT ? 64 : pl.bt / 2);
    if (!st) st = kernels.check();
    if (!st) st = wg::ensure_smem(kernels.product, wg::kLinSmem);
    const long long segments = (long long)ka.segments * ka.batch + kb.segments;
    if (!st && segments > 0)
        st = launch("linear_pack_kernel launch", wg::linear_pack_kernel, dim3((unsigned)std::min<long long>((segments + 7) / 8, 8LL * num_sms())),
                    dim3(256), s, ka, kb, offsets, (int)(q.offset_bits == 64), q.tokens);
    if (!st && sums) st = columns_launch(*sums, pl, s);
    if (st) return st;
    wg::LinParams g = {};
    g.t = tail;
    if (few) g.few = *few;
    g.experts = q.experts, g.offsets = offsets, g.offsets64 = q.offset_bits == 64, g.tokens = q.tokens;
    g.M = pl.M, g.N = pl.N, g.kb = pl.kb, g.bf16 = bf16;
    g.chunk = lin_chunk(q);
    g.bt = pl.bt, g.stages = pl.stages, g.stage_bytes = pl.stage_bytes, g.split = pl.split, g.pairs = pl.pairs;
    const unsigned im = (unsigned)(pl.M + 255) / 256;
    g.by_bt = wg::fast_div((unsigned)pl.bt), g.by_im = wg::fast_div(im), g.by_8im = wg::fast_div(8 * im);
    g.by_per = wg::fast_div(im * (unsigned)((std::max(pl.N, 1) + pl.bt - 1) / pl.bt));
    g.part = reinterpret_cast<float*>(ws + pl.off_part), g.ldp = pl.ldp, g.part_rows = pl.part_rows;
    const long long items = g.part_rows * (g.ldp / 8);
    g.join_blocks = (int)std::min<long long>((items + wg::kJoinBlock - 1) / wg::kJoinBlock, 16LL * num_sms());
    if (joined && joined->part) {
        // In the last launch, where one round of its blocks does it (64 experts' 2048 columns are 512 units).
        wg::SumParams m = *joined;
        const int ne = std::max(q.experts, 1);
        plan_join(&m, ne, pl.sum_chunks, pl.split > 1 ? wg::kJoinBlock : wg::kJoinThreads);
        if (m.units <= (pl.split > 1 ? 4 * num_sms() : 2 * pl.pairs)) g.sums = m, joined->part = nullptr;
    }
    return product_launch(pl, kernels, ma, mb, g, s);
}

template <int XR, int FG, int VEC>
int rows_launch(const wg::RowsParams& g, bool bf16, cudaStream_t s)
{
    const long long passes = std::max(1LL, std::min(g.tokens, std::max(g.experts, 1) + g.tokens / (8 * XR)));  // at most
    const long long items = passes * ((g.M + 8 * FG - 1) / (8 * FG));
    // (What an SM holds: 4 rows of 16 experts' 1024 x 4096 12.0 us against 12.6 with four times that.)
    const dim3 grid((unsigned)std::min<long long>(items, 2LL * num_sms()));
    return launch("linear_rows_kernel launch", bf16 ? wg::linear_rows_kernel<XR, FG, true, VEC> : wg::linear_rows_kernel<XR, FG, false, VEC>,
                  grid, dim3(wg::kRowsThreads), s, g);
}
// Rows of a pass by eight, columns of a block by eight, elements of an access.
struct RowsShape {
    int xr, fg, vec;
};
RowsShape rows_shape(const wg_linear_problem& q, const void* x, const void* w)
{
    const auto rows_of = [&](int v) {
        return q.in % v == 0 && q.ld_in % v == 0 && q.ld_weight % v == 0 && (q.experts <= 1 || q.weight_stride % v == 0) &&
               aligned_to(x, 2 * v) && aligned_to(w, 2 * v);
    };
    const bool one = q.tokens <= 8 || q.experts > 1;
    const long long used = std::min<long long>(std::max(q.experts, 1), q.tokens);
    const auto many = [&](int columns) { return 2 * ((q.out + columns - 1) / columns) * used >= 3LL * num_sms(); };  // CTAs
    // Sixteen rows per pass of one weight matrix only (64 of 8 experts', 8 each, 33 us against 26).
    // 32 columns of the result per CTA where those are enough CTAs (8192 x 8192 23.5 us against 24.7
    // with 16, 4096 x 16384 25.1 against 27.4, 8000 rows of 999 9.4 against 11.3), else 16 (4096 x 4096 9.2
    // against 11.7).
    if (rows_of(8)) return {one ? 1 : 2, one && many(32) ? 4 : 2, 8};
    if (rows_of(2)) return {one ? 1 : 2, 2, 2};
    return {one ? 1 : 2, !one ? 2 : many(32) ? 4 : many(16) ? 2 : 1, 1};
}

int rows_run(const LinPlan& pl, const void* offsets, const void* x, const void* w, const wg::LayerTail& tail, cudaStream_t s)
{
    const wg_linear_problem& q = pl.p;
    wg::RowsParams g = {};
    g.t = tail, g.experts = q.experts, g.offsets64 = q.offset_bits == 64, g.offsets = offsets, g.tokens = q.tokens;
    g.x = x, g.w = w, g.ldx = q.ld_in, g.ldw = q.ld_weight, g.wstride = q.weight_stride, g.K = q.in, g.M = q.out;
    const bool bf16 = q.in_dtype == WG_BF16;
    const RowsShape h = rows_shape(q, x, w);
    if (h.vec == 8) return h.xr == 2 ? rows_launch<2, 2, 8>(g, bf16, s) : h.fg == 4 ? rows_launch<1, 4, 8>(g, bf16, s) : rows_launch<1, 2, 8>(g, bf16, s);
    if (h.vec == 2) return h.xr == 2 ? rows_launch<2, 2, 2>(g, bf16, s) : rows_launch<1, 2, 2>(g, bf16, s);
    if (h.xr == 2) return rows_launch<2, 2, 1>(g, bf16, s);
    return h.fg == 4 ? rows_launch<1, 4, 1>(g, bf16, s) : h.fg == 2 ? rows_launch<1, 2, 1>(g, bf16, s) : rows_launch<1, 1, 1>(g, bf16, s);
}

int lin_offsets(const LinPlan& pl, const void* offsets)
{
    if ((pl.p.experts > 0) != (offsets != nullptr))
        return set_err(WG_ERR_INVALID_ARGUMENT, "offsets must be given with experts, and NULL without");
    return WG_OK;
}

// ---------------------------------------------------------------- activation alone
struct ActPlan {
    wg_activation_problem p;
    int cx_log, chunk;
    long long chunks;
    size_t bytes;
};

int act_plan(const wg_activation_problem* p, ActPlan* pl)
{
    if (!p) return set_err(WG_ERR_INVALID_ARGUMENT, "problem is NULL");
    if (p->tokens < 0 || p->dim < 1) return set_err(WG_ERR_INVALID_ARGUMENT, "tokens must be at least 0 and dim at least 1");
    if (p->tokens > kMaxTokens || p->dim > kMaxFeatures)
        return set_err(WG_ERR_NOT_SUPPORTED, "tokens up to 2^31-65536 and dim up to 2^20 are supported");
    if (!dtype_ok(p->in_dtype) || !dtype_ok(p->out_dtype) || !dtype_ok(p->bias_dtype))
        return set_err(WG_ERR_INVALID_ARGUMENT, "in_dtype, out_dtype and bias_dtype must be WG_FP32, WG_BF16 or WG_FP16");
    const int st = check_factors(p->activation, p->dropout, p->counter);
    if (st) return st;
    pl->p = *p;
    wg_activation_problem& q = pl->p;
    const long long far = kMaxSpan / std::max(q.tokens, 1LL);
    for (long long* ld : {&q.ld_x, &q.ld_y, &q.ld_residual, &q.ld_dx}) {
        if (*ld == 0) *ld = q.dim;
        if (*ld < q.dim) return set_err(WG_ERR_INVALID_ARGUMENT, "a row stride must be 0 or at least dim");
        if (*ld > far) return set_err(WG_ERR_INVALID_ARGUMENT, "a row stride is larger than any memory");
    }
    // Threads side by side (at most 32, 256 columns), and rows of a block: some 12 blocks per SM, so that their
    // ends even out, of at least one row per thread.
    const int groups = (q.dim + 7) / 8;
    pl->cx_log = std::min(5, log2_floor(groups) + ((groups & (groups - 1)) ? 1 : 0));
    const long long cols = (groups + (1 << pl->cx_log) - 1) >> pl->cx_log, ny = wg::kActThreads >> pl->cx_log;
    const long long want = std::max(1LL, 12LL * num_sms() / cols);
    long long rows = std::max(ny, (q.tokens + want - 1) / want);
    rows = (rows + ny - 1) / ny * ny;
    if (rows > ny) rows = (rows + 4 * ny - 1) / (4 * ny) * (4 * ny);  // (whole rounds of the rows in flight)
    rows = std::max(rows, ((q.tokens + 65534) / 65535 + ny - 1) / ny * ny);
    pl->chunk = (int)rows;
    pl->chunks = std::max(1LL, (q.tokens + rows - 1) / rows);
    pl->bytes = up256((size_t)pl->chunks * q.dim * 4);
    return WG_OK;
}

template <bool BWD, int MODE>
int act_launch_mode(const ActPlan& pl, const wg::ActParams& g, cudaStream_t s)
{
    const int groups = (pl.p.dim + 7) / 8;
    return launch("activation_kernel launch", wg::activation_kernel<BWD, MODE>,
                  dim3((unsigned)((groups + (1 << pl.cx_log) - 1) >> pl.cx_log), (unsigned)pl.chunks), dim3(wg::kActThreads), s, g);
}
template <bool BWD>
int act_launch(const ActPlan& pl, const wg::ActParams& g, cudaStream_t s)
{
    const bool half = g.t.y_dtype != 2 && (!g.x || g.x_dtype != 2) && (!BWD || g.dy_dtype != 2);
    const bool wide = (!g.x || g.vec_x) && (!BWD || g.vec_dy) && (!g.t.y || (g.t.vec & wg::kVecY)) && (!g.t.res || (g.t.vec & wg::kVecRes));
    if (half && wide) return act_launch_mode<BWD, wg::kActWide>(pl, g, s);
    return half && pl.cx_log == 5 ? act_launch_mode<BWD, wg::kActShifted>(pl, g, s) : act_launch_mode<BWD, wg::kActAny>(pl, g, s);
}

wg::ActParams act_params(const ActPlan& pl, const void* x, const void* bias)
{
    const wg_activation_problem& q = pl.p;
    wg::ActParams g = {};
    g.rows = q.tokens, g.dim = q.dim, g.x = x, g.ldx = q.ld_x, g.x_dtype = q.in_dtype;
    g.vec_x = vec_rows(x, q.ld_x, q.dim, esize(q.in_dtype));
    g.cx_log = pl.cx_log, g.chunk = pl.chunk;
    g.t.bias = bias, g.t.bias_dtype = q.bias_dtype, g.t.act = q.activation;
    if (vec_rows(bias, 0, q.dim, esize(q.bias_dtype))) g.t.vec |= wg::kVecBias;
    set_dropout(&g.t, q.dropout, q.seed, q.offset, q.counter);
    return g;
}

}  // namespace

extern "C" {

int wg_linear_workspace_size(const wg_linear_problem* p, wg_linear_call call, size_t* bytes)
{
    if (!bytes) return set_err(WG_ERR_INVALID_ARGUMENT, "bytes is NULL");
    LinPlan pl;
    const int st = lin_plan(p, call, &pl);
    if (!st) *bytes = pl.bytes;
    return st;
}

int wg_linear_plan_string(const wg_linear_problem* p, wg_linear_call call, char* buf, size_t n)
{
    if (!buf || n == 0) return set_err(WG_ERR_INVALID_ARGUMENT, "buffer is NULL or empty");
    LinPlan pl;
    const int st = lin_plan(p, call, &pl);
    if (st) return st;
    if (pl.few) {
        const RowsShape h = rows_shape(pl.p, nullptr, nullptr);  // (for bases on 16 bytes)
        snprintf(buf, n, "kernel=linear_rows call=forward rows=%d columns=%d access=%d ws=%zu", 8 * h.xr, 8 * h.fg, h.vec, pl.bytes);
        return WG_OK;
    }
    static const char* const kNames[3] = {"forward", "bwd_data", "bwd_weight"};
    snprintf(buf, n, "kernel=linear_product call=%s columns=%d rows=%d split=%d chunks=%lld stages=%d pairs=%d pack=%d%d smem=%d ws=%zu",
             kNames[pl.call], 256, pl.bt, pl.split, pl.chunks, pl.stages, pl.pairs, pl.pack_a, pl.pack_b, wg::kLinSmem, pl.bytes);
    return WG_OK;
}

int wg_linear(const wg_linear_problem* p, const void* offsets, const void* x, const void* w, const void* bias, const void* residual,
              void* y, void* z, void* workspace, size_t ws_bytes, void* stream)
{
    LinPlan pl;
    int st = lin_plan(p, WG_LINEAR_FORWARD, &pl);
    if (st || (st = lin_offsets(pl, offsets))) return st;
    const wg_linear_problem& q = pl.p;
    if (q.tokens > 0 && (!x || !w || !y)) return set_err(WG_ERR_INVALID_ARGUMENT, "x, w and y must be non-NULL device pointers");
    const int ne = std::max(q.experts, 1), ie = esize(q.in_dtype), oe = esize(q.out_dtype), be = esize(q.bias_dtype);
    const Tensor t[] = {{"y", y, q.tokens, q.out, q.ld_out, oe, 1, 0},
                        {"z", z, q.tokens, q.out, q.ld_z, ie, 1, 0},
                        {"residual", residual, q.tokens, q.out, q.ld_residual, oe, 1, 0},
                        {"x", x, q.tokens, q.in, q.ld_in, ie, 1, 0},
                        {"w", w, q.out, q.in, q.ld_weight, ie, ne, q.weight_stride},
                        {"bias", bias, ne, q.out, q.out, be, 1, 0},
                        {"offsets", offsets, 1, ne + 1, ne + 1, q.offset_bits / 8, 1, 0},
                        {"counter", q.counter, 1, 1, 1, 8, 1, 0}};
    if ((st = check_tensors(t, 8, 2, 0, 2))) return st;
    if ((st = check_workspace(pl.bytes, workspace, ws_bytes))) return st;
    if (q.tokens == 0) return WG_OK;
    wg::LayerTail g = {};
    g.y = y, g.y_dtype = q.out_dtype, g.ldy = q.ld_out, g.res = residual, g.ldr = q.ld_residual;
    g.z = z, g.z_dtype = q.in_dtype, g.ldz = q.ld_z, g.act = q.activation;
    g.bias = bias, g.bias_dtype = q.bias_dtype, g.bias_stride = q.out;
    if (vec_rows(y, q.ld_out, q.out, oe)) g.vec |= wg::kVecY;
    if (pair_rows(y, q.ld_out, q.out, oe)) g.vec |= wg::kPairY;
    if (vec_rows(z, q.ld_z, q.out, ie)) g.vec |= wg::kVecZ;
    if (pair_rows(z, q.ld_z, q.out, ie)) g.vec |= wg::kPairZ;
    if (vec_rows(residual, q.ld_residual, q.out, oe)) g.vec |= wg::kVecRes;
    if (pair_rows(residual, q.ld_residual, q.out, oe)) g.vec |= wg::kPairRes;
    if (vec_rows(bias, q.out, q.out, be)) g.vec |= wg::kVecBias;
    set_dropout(&g, q.dropout, q.seed, q.offset, q.counter);
    if (pl.few) return rows_run(pl, offsets, x, w, g, static_cast<cudaStream_t>(stream));
    return lin_run(pl, offsets, {w, q.out, q.in, q.ld_weight, ne, q.weight_stride}, {x, q.tokens, q.in, q.ld_in, 1, 0}, g,
                   static_cast<char*>(workspace), static_cast<cudaStream_t>(stream));
}

int wg_linear_bwd_data(const wg_linear_problem* p, const void* offsets, const void* dy, const void* w, const void* z,
                       const void* residual, void* dx, void* workspace, size_t ws_bytes, void* stream)
{
    LinPlan pl;
    int st = lin_plan(p, WG_LINEAR_BWD_DATA, &pl);
    if (st || (st = lin_offsets(pl, offsets))) return st;
    const wg_linear_problem& q = pl.p;
    if (q.activation == WG_ACT_NONE) z = nullptr;
    if (q.tokens > 0 && (!dy || !w || !dx || (q.activation != WG_ACT_NONE && !z)))
        return set_err(WG_ERR_INVALID_ARGUMENT, "dy, w, dx, and z of an activation, must be non-NULL device pointers");
    const int ne = std::max(q.experts, 1), ie = esize(q.in_dtype), oe = esize(q.out_dtype);
    const Tensor t[] = {{"dx", dx, q.tokens, q.in, q.ld_in, oe, 1, 0},
                        {"residual", residual, q.tokens, q.in, q.ld_residual, oe, 1, 0},
                        {"z", z, q.tokens, q.in, q.ld_z, ie, 1, 0},
                        {"dy", dy, q.tokens, q.out, q.ld_out, ie, 1, 0},
                        {"w", w, q.out, q.in, q.ld_weight, ie, ne, q.weight_stride},
                        {"offsets", offsets, 1, ne + 1, ne + 1, q.offset_bits / 8, 1, 0},
                        {"counter", q.counter, 1, 1, 1, 8, 1, 0}};
    if ((st = check_tensors(t, 7, 1, 0, 1))) return st;
    if ((st = check_workspace(pl.bytes, workspace, ws_bytes))) return st;
    if (q.tokens == 0) return WG_OK;
    wg::LayerTail g = {};
    g.y = dx, g.y_dtype = q.out_dtype, g.ldy = q.ld_in, g.res = residual, g.ldr = q.ld_residual;
    g.z = const_cast<void*>(z), g.z_dtype = q.in_dtype, g.ldz = q.ld_z, g.act = q.activation;
    if (vec_rows(dx, q.ld_in, q.in, oe)) g.vec |= wg::kVecY;
    if (pair_rows(dx, q.ld_in, q.in, oe)) g.vec |= wg::kPairY;
    if (vec_rows(z, q.ld_z, q.in, ie)) g.vec |= wg::kVecZ;
    if (pair_rows(z, q.ld_z, q.in, ie)) g.vec |= wg::kPairZ;
    if (vec_rows(residual, q.ld_residual, q.in, oe)) g.vec |= wg::kVecRes;
    if (pair_rows(residual, q.ld_residual, q.in, oe)) g.vec |= wg::kPairRes;
    set_dropout(&g, q.dropout, q.seed, q.offset, q.counter);
    return lin_run(pl, offsets, {w, q.out, q.in, q.ld_weight, ne, q.weight_stride}, {dy, q.tokens, q.out, q.ld_out, 1, 0}, g,
                   static_cast<char*>(workspace), static_cast<cudaStream_t>(stream));
}

int wg_linear_bwd_weight(const wg_linear_problem* p, const void* offsets, const void* x, const void* dy, void* dw, void* dbias,
                         int accumulate, void* workspace, size_t ws_bytes, void* stream)
{
    LinPlan pl;
    int st = lin_plan(p, WG_LINEAR_BWD_WEIGHT, &pl);
    if (st || (st = lin_offsets(pl, offsets))) return st;
    const wg_linear_problem& q = pl.p;
    if ((q.tokens > 0 && (!x || !dy)) || !dw) return set_err(WG_ERR_INVALID_ARGUMENT, "x, dy and dw must be non-NULL device pointers");
    const int ne = std::max(q.experts, 1), ie = esize(q.in_dtype), oe = esize(q.out_dtype);
    const Tensor t[] = {{"dw", dw, q.out, q.in, q.ld_weight, oe, ne, q.weight_stride},
                        {"dbias", dbias, ne, q.out, q.out, esize(q.bias_dtype), 1, 0},
                        {"x", x, q.tokens, q.in, q.ld_in, ie, 1, 0},
                        {"dy", dy, q.tokens, q.out, q.ld_out, ie, 1, 0},
                        {"offsets", offsets, 1, ne + 1, ne + 1, q.offset_bits / 8, 1, 0}};
    if ((st = check_tensors(t, 5, 2, -1, -1))) return st;
    if ((st = check_workspace(pl.bytes, workspace, ws_bytes))) return st;
    char* ws = static_cast<char*>(workspace);
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    wg::LayerTail g = {};
    g.y = dw, g.y_dtype = q.out_dtype, g.ldy = q.ld_weight, g.y_stride = q.weight_stride;
    g.gain = 1.f;
    if (accumulate) g.res = dw, g.ldr = q.ld_weight;
    if (vec_rows(dw, q.ld_weight, q.in, oe, ne > 1 ? q.weight_stride : 0)) g.vec |= wg::kVecY | wg::kVecRes;
    if (pair_rows(dw, q.ld_weight, q.in, oe, ne > 1 ? q.weight_stride : 0)) g.vec |= wg::kPairY | wg::kPairRes;
    if (!dbias) return lin_run(pl, offsets, {x, q.tokens, q.in, q.ld_in, 1, 0}, {dy, q.tokens, q.out, q.ld_out, 1, 0}, g, ws, s);
    const bool vec = vec_rows(dy, q.ld_out, q.out, ie);
    // Few rows: within the product, 64 columns and every row of an expert per CTA.
    wg::FewSums few = {};
    few.across = (q.out + 63) / 64, few.units = ne * few.across;
    if (q.tokens <= kFewSums && few.units <= 4 * num_sms()) {
        few.dy = dy, few.ld = q.ld_out, few.out = dbias, few.dtype = q.in_dtype, few.out_dtype = q.bias_dtype;
        few.accumulate = accumulate != 0, few.vec = vec;
        return lin_run(pl, offsets, {x, q.tokens, q.in, q.ld_in, 1, 0}, {dy, q.tokens, q.out, q.ld_out, 1, 0}, g, ws, s, &few);
    }
    wg::ColumnParams c = {};
    c.dy = dy, c.tokens = q.tokens, c.ld = q.ld_out, c.N = q.out, c.dtype = q.in_dtype;
    c.experts = q.experts, c.offsets64 = q.offset_bits == 64, c.offsets = offsets, c.chunk = pl.sum_rows;
    c.part = reinterpret_cast<float*>(ws + pl.off_sum), c.first = reinterpret_cast<int*>(ws + pl.off_first);
    const int groups = (q.out + 7) / 8;
    c.cx_log = std::min(5, log2_floor(groups) + ((groups & (groups - 1)) ? 1 : 0));
    wg::SumParams m = {};
    m.part = c.part, m.out = dbias, m.dim = q.out, m.dtype = q.bias_dtype, m.accumulate = accumulate != 0, m.first = c.first;
    st = lin_run(pl, offsets, {x, q.tokens, q.in, q.ld_in, 1, 0}, {dy, q.tokens, q.out, q.ld_out, 1, 0}, g, ws, s, nullptr, &c, &m);
    return st || !m.part ? st : join_columns(m, ne, pl.sum_chunks, s);
}

int wg_activation_workspace_size(const wg_activation_problem* p, size_t* bytes)
{
    if (!bytes) return set_err(WG_ERR_INVALID_ARGUMENT, "bytes is NULL");
    ActPlan pl;
    const int st = act_plan(p, &pl);
    if (!st) *bytes = pl.bytes;
    return st;
}

int wg_activation(const wg_activation_problem* p, const void* x, const void* bias, const void* residual, void* y, void* stream)
{
    ActPlan pl;
    int st = act_plan(p, &pl);
    if (st) return st;
    const wg_activation_problem& q = pl.p;
    if (q.tokens > 0 && (!x || !y)) return set_err(WG_ERR_INVALID_ARGUMENT, "x and y must be non-NULL device pointers");
    const int ie = esize(q.in_dtype), oe = esize(q.out_dtype);
    // (Types of one size are still different types.)
    const Tensor t[] = {{"y", y, q.tokens, q.dim, q.ld_y, oe, 1, 0},
                        {"x", x, q.tokens, q.dim, q.ld_x, ie, 1, 0},
                        {"residual", residual, q.tokens, q.dim, q.ld_residual, oe, 1, 0},
                        {"bias", bias, 1, q.dim, q.dim, esize(q.bias_dtype), 1, 0},
                        {"counter", q.counter, 1, 1, 1, 8, 1, 0}};
    if ((st = check_tensors(t, 5, 1, 0, q.in_dtype == q.out_dtype ? 1 : 2, 2))) return st;
    if (q.tokens == 0) return WG_OK;
    wg::ActParams g = act_params(pl, x, bias);
    g.t.y = y, g.t.y_dtype = q.out_dtype, g.t.ldy = q.ld_y, g.t.res = residual, g.t.ldr = q.ld_residual;
    if (vec_rows(y, q.ld_y, q.dim, oe)) g.t.vec |= wg::kVecY;
    if (vec_rows(residual, q.ld_residual, q.dim, oe)) g.t.vec |= wg::kVecRes;
    return act_launch<false>(pl, g, static_cast<cudaStream_t>(stream));
}

int wg_activation_bwd(const wg_activation_problem* p, const void* dy, const void* x, const void* bias, void* dx, void* dbias,
                      void* workspace, size_t ws_bytes, void* stream)
{
    ActPlan pl;
    int st = act_plan(p, &pl);
    if (st) return st;
    const wg_activation_problem& q = pl.p;
    if (q.activation == WG_ACT_NONE) x = nullptr;
    if ((q.tokens > 0 && (!dy || (q.activation != WG_ACT_NONE && !x))) || (!dx && !dbias))
        return set_err(WG_ERR_INVALID_ARGUMENT, "dy, x of an activation, and one of dx and dbias, must be non-NULL device pointers");
    const int ie = esize(q.in_dtype), oe = esize(q.out_dtype), be = esize(q.bias_dtype);
    const Tensor t[] = {{"dx", dx, q.tokens, q.dim, q.ld_dx, ie, 1, 0},
                        {"dbias", dbias, 1, q.dim, q.dim, be, 1, 0},
                        {"dy", dy, q.tokens, q.dim, q.ld_y, oe, 1, 0},
                        {"x", x, q.tokens, q.dim, q.ld_x, ie, 1, 0},
                        {"bias", bias, 1, q.dim, q.dim, be, 1, 0},
                        {"counter", q.counter, 1, 1, 1, 8, 1, 0}};
    if ((st = check_tensors(t, 6, 2, 0, q.in_dtype == q.out_dtype ? 2 : 3, 3))) return st;
    if (dbias && (st = check_workspace(pl.bytes, workspace, ws_bytes))) return st;
    if (q.tokens == 0 && !dbias) return WG_OK;
    wg::ActParams g = act_params(pl, x, bias);
    g.t.y = dx, g.t.y_dtype = q.in_dtype, g.t.ldy = q.ld_dx;
    if (vec_rows(dx, q.ld_dx, q.dim, ie)) g.t.vec |= wg::kVecY;
    g.dy = dy, g.lddy = q.ld_y, g.dy_dtype = q.out_dtype, g.vec_dy = vec_rows(dy, q.ld_y, q.dim, oe);
    g.part = dbias ? static_cast<float*>(workspace) : nullptr;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if ((st = act_launch<true>(pl, g, s)) || !dbias) return st;
    wg::SumParams m = {};
    m.part = g.part, m.out = dbias, m.dim = q.dim, m.dtype = q.bias_dtype, m.chunks = (int)pl.chunks;
    return join_columns(m, 1, pl.chunks, s);
}

}  // extern "C"
