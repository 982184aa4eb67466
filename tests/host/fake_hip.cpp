// Stands in for the HIP runtime's launch path (loaded before it, for all to see):
// launches are not made, their grids are recorded.
#include <cstddef>
#include <cstdint>

namespace {
struct Dim { uint32_t x, y, z; };
thread_local Dim grid_, block_;
thread_local size_t lds_;
thread_local void* stream_;
uint64_t launches, most_threads, most_groups, most_lds;
uint32_t most_block, empty, most_yz;
}  // namespace

extern "C" {
int __hipPushCallConfiguration(Dim g, Dim b, size_t lds, void* s) {
    grid_ = g;
    block_ = b;
    lds_ = lds;
    stream_ = s;
    return 0;
}
int __hipPopCallConfiguration(Dim* g, Dim* b, size_t* lds, void** s) {
    *g = grid_;
    *b = block_;
    *lds = lds_;
    *s = stream_;
    return 0;
}
int hipLaunchKernel(const void*, Dim g, Dim b, void**, size_t lds, void*) {
    ++launches;
    auto top = [](auto& m, auto v) { m = v > m ? decltype(m + m)(v) : m; };
    const uint32_t block = b.x * b.y * b.z;
    const uint64_t groups = uint64_t(g.x) * g.y * g.z;
    if (groups == 0 || block == 0) ++empty;
    top(most_threads, uint64_t(g.x) * b.x > uint64_t(g.y) * b.y ? uint64_t(g.x) * b.x : uint64_t(g.y) * b.y);
    top(most_groups, groups);
    top(most_block, block);
    top(most_yz, g.y > g.z ? g.y : g.z);
    top(most_lds, uint64_t(lds));
    return 0;
}
int hipGetLastError() { return 0; }
// launches, empty ones, most threads along an axis, most workgroups, most threads of a
// workgroup, most workgroups along y and z; and starts again
void fake_hip_take(uint64_t* out) {
    const uint64_t v[6] = {launches, empty, most_threads, most_groups, most_block, most_yz};
    for (int i = 0; i < 6; ++i) out[i] = v[i];
    launches = most_threads = most_groups = most_lds = 0;
    most_block = empty = most_yz = 0;
}
}
