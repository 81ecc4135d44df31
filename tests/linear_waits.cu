// linear_waits.cu -- the scans of the gated linear recurrence with their first place left out, so that the wait for it runs
// out: for a test of what the kernels do then.  Channels of fp32, gates per channel; every wait has a limit of `cycles`.
#include "gdn_linear_column_backward.cuh"

using namespace gdn;
using namespace gdn::linear;

namespace {

constexpr int kPlaces = 3, kStages = 2;  // of columns: time segments, and stages of each
using Forward = Column<32, kForwardWarps, 8, kForwardGroups, true>;
using Backward = Column<32, 8, backward_run<float, kPerChannel>(), backward_groups<float, float, kPerChannel>(), true>;

template <class Kernel>
cudaError_t launch(Kernel kernel, unsigned blocks, int threads, int smem, const LinearParams& p, const Segments& seg, int box,
                   cudaStream_t stream) {
    ColumnMaps maps{};
    if (!encode_rows(&maps.x, p.x, p.x_dt, p.x_stride, p.C, p.T, 32, box) ||
        !encode_rows(&maps.a, p.a, p.gate_dt, p.a_stride, p.C, p.T, 32, box) ||
        (p.dy && !encode_rows(&maps.dy, p.dy, p.x_dt, p.dy_stride, p.C, p.T, 32, box)))
        return cudaErrorInvalidValue;
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    kernel<<<blocks, threads, smem, stream>>>(p, seg, maps);
    return cudaGetLastError();
}

}  // namespace

extern "C" {

// Tokens of a batch of kPlaces segments, or of as many tiles.
int waits_tokens(int column, int backward) {
    if (!column) return kPlaces * kTile;
    return kPlaces * kStages * (backward ? Backward::kTokens : Forward::kTokens);
}

// x, a, y (or dx, da) [waits_tokens][C], C a multiple of 128; cu [3]: two sequences; state [2][C] (or d_initial); tile_states
// as the forward pass saves them.  workspace: zeros, 64 KB or more.  Returns a CUDA error.
int waits_run(int column, int backward, const float* x, const float* a, const int* cu, int C, float* y, float* da, float* state,
              float* tile_states, int* status, void* workspace, int64_t cycles, void* stream) {
    LinearParams p{};
    p.x = x;
    p.a = a;
    p.x_stride = p.a_stride = p.y_stride = p.dy_stride = p.dx_stride = p.da_stride = p.state_stride = C;
    p.D = p.C = C;
    p.H = p.gate_div = 1;
    p.x_dt = p.gate_dt = p.state_dt = GDN_DTYPE_F32;
    p.cu_seqlens = cu;
    p.N = 2;
    p.T = waits_tokens(column, backward);
    p.status = status;
    p.tile_states = tile_states;
    if (backward) {
        p.dy = x;
        p.dx = y;
        p.da = da;
        p.initial_state = state + 2 * C;
        p.d_initial = state;
    } else {
        p.y = y;
        p.output_state = state;
    }
    uint8_t* ws = static_cast<uint8_t*>(workspace);
    Segments seg{};
    seg.first = seg.stages = kStages;
    ScanSpace& s = seg.space;
    s.nt = kPlaces;
    s.blocks = static_cast<uint32_t>(column ? C / 32 : C / 128);
    s.wait_cycles = cycles;
    s.ticket = reinterpret_cast<uint32_t*>(ws);
    s.flags = reinterpret_cast<uint32_t*>(ws + 256);
    s.pairs = reinterpret_cast<float2*>(ws + 4096);
    s.known = reinterpret_cast<float*>(ws + 4096 + 8 * kPlaces * C);
    s.exponents = reinterpret_cast<int32_t*>(ws + 4096 + 12 * kPlaces * C);
    if (C % 128 || 4 * kPlaces * 4 * s.blocks > 4096 - 256 || 4096 + 16 * kPlaces * C > 65536) return cudaErrorInvalidValue;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    const uint32_t skipped = s.blocks;  // the first place's tickets are gone
    cudaError_t e = cudaMemcpyAsync(s.ticket, &skipped, 4, cudaMemcpyHostToDevice, st);
    if (e != cudaSuccess) return e;
    const unsigned blocks = (kPlaces - 1) * s.blocks;
    if (column && backward)
        return launch(gdn_linear_column_backward_kernel<float, float, kPerChannel, false, Backward>, blocks, Backward::kThreads,
                      BackwardShape<float, float, kPerChannel, false, Backward>::kSmem, p, seg, StageArray<float, Backward>::kBox, st);
    if (column)
        return launch(gdn_linear_column_forward_kernel<float, float, kPerChannel, false, Forward>, blocks, Forward::kThreads,
                      ForwardShape<float, float, kPerChannel, false, Forward>::kSmem, p, seg, StageArray<float, Forward>::kBox, st);
    if (backward)
        gdn_linear_backward_kernel<float, float, true, false, false><<<blocks, kThreads, 0, st>>>(p, s);
    else
        gdn_linear_forward_kernel<float, float, true, false, false><<<blocks, kThreads, 0, st>>>(p, s);
    return cudaGetLastError();
}
}
