// Test harness: the launch entry points of the HIP runtime, replaced by ones
// that write down what would be launched (kernel, blocks, threads per block)
// and launch nothing. Loaded in front of the library in a process of its own,
// it shows on a machine without a GPU which kernels a call takes and how many
// of their blocks. Test infrastructure only; built with g++, no HIP.
#include <cstdint>
#include <map>
#include <string>
#include <vector>

namespace {

struct Dim3 {
    uint32_t x, y, z;
};
struct Launch {
    std::string kernel;
    Dim3 grid, block;
};
std::map<const void*, std::string>& names() {
    static std::map<const void*, std::string> m;
    return m;
}
std::vector<Launch> launches;
Dim3 next_grid, next_block;
size_t next_lds;
void* next_stream;

}  // namespace

extern "C" {

void __hipRegisterFunction(void**, const void* host, char*, const char* device, unsigned, void*, void*, void*, void*,
                           int*) {
    names()[host] = device;
}

int __hipPushCallConfiguration(Dim3 grid, Dim3 block, size_t lds, void* stream) {
    next_grid = grid;
    next_block = block;
    next_lds = lds;
    next_stream = stream;
    return 0;
}

int __hipPopCallConfiguration(Dim3* grid, Dim3* block, size_t* lds, void** stream) {
    *grid = next_grid;
    *block = next_block;
    *lds = next_lds;
    *stream = next_stream;
    return 0;
}

int hipLaunchKernel(const void* host, Dim3 grid, Dim3 block, void**, size_t, void*) {
    launches.push_back(Launch{names()[host], grid, block});
    return 0;
}

int hipGetLastError() { return 0; }

// Launches since the last ll_clear: their number, and launch i's kernel (its
// symbol) and dims: grid x, y, z, block x, y, z.
int ll_count() { return (int)launches.size(); }
const char* ll_launch(int i, uint32_t* dims) {
    const Launch& l = launches[(size_t)i];
    const uint32_t d[6] = {l.grid.x, l.grid.y, l.grid.z, l.block.x, l.block.y, l.block.z};
    for (int k = 0; k < 6; ++k) dims[k] = d[k];
    return l.kernel.c_str();
}
void ll_clear() { launches.clear(); }

}  // extern "C"
