// Which kernels a call of the 8-bit experts launches, without a GPU (test infrastructure): the
// library's host code is linked with the launch functions below, which note a kernel's name
// instead of running it.  First line: every kernel of the library, then one line for each call
// read from stdin, with its kernels in order and their grids; names are parted by tabs.
//     gemv E grouped N M K ldx ldy s_dtype y_dtype w_offset x_offset
//     sort T top_k E H x_dtype        unsort T top_k H r_dtype y_dtype
//     grad T top_k H y_dtype r_dtype  swiglu N I g_dtype out_dtype
#include <cxxabi.h>
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <iostream>
#include <map>
#include <sstream>
#include <string>

#include "../../include/seedmm.h"

static std::map<const void*, std::string>& kernels() {
    static std::map<const void*, std::string> k;
    return k;
}
static std::string launched;
static dim3 grid_now, block_now;

// "k_name<1, 2>" of the device's symbol
static std::string short_name(const char* symbol) {
    int status = 0;
    char* s = abi::__cxa_demangle(symbol, nullptr, nullptr, &status);
    std::string n = status == 0 ? s : symbol;
    free(s);
    const size_t at = n.find("::k_");
    if (at != std::string::npos) n = n.substr(at + 2);
    return n.substr(0, n.find('('));
}

extern "C" {
void** __hipRegisterFatBinary(const void*) {
    static void* none[1];
    return none;
}
void __hipUnregisterFatBinary(void**) {}
void __hipRegisterFunction(void**, const void* host, char*, const char* device, unsigned, void*, void*, void*, void*, int*) {
    kernels()[host] = short_name(device);
}
hipError_t __hipPushCallConfiguration(dim3 grid, dim3 block, size_t, hipStream_t) {
    grid_now = grid;
    block_now = block;
    return hipSuccess;
}
hipError_t __hipPopCallConfiguration(dim3* grid, dim3* block, size_t* shared, hipStream_t* st) {
    *grid = grid_now;
    *block = block_now;
    *shared = 0;
    *st = nullptr;
    return hipSuccess;
}
hipError_t hipLaunchKernel(const void* host, dim3 grid, dim3, void**, size_t, hipStream_t) {
    launched += "\t" + kernels().at(host) + " " + std::to_string(grid.x);
    return hipSuccess;
}
hipError_t hipGetLastError() { return hipSuccess; }
}

int main() {
    char* F = (char*)(uintptr_t)0x100000;    // no kernel runs: never dereferenced
    std::string all;
    for (auto& k : kernels()) all += "\t" + k.second;
    std::cout << all << "\n";
    std::string line, op;
    while (std::getline(std::cin, line)) {
        std::istringstream in(line);
        in >> op;
        int64_t v[12] = {};
        for (int i = 0; i < 12 && in >> v[i]; ++i) {}
        int status = 0;
        launched.clear();
        if (op == "gemv")
            status = seedmm_i8_gemv((int8_t*)F + v[9], F, (int)v[7], (int)v[0], v[1] ? (int32_t*)F : nullptr,
                                    (int8_t*)F + v[10], v[5], (float*)F, F, (int)v[8], v[6], (int)v[3], (int)v[4], (int)v[2], nullptr);
        else if (op == "sort")
            status = seedmm_moe_sort((int32_t*)F, (int)v[0], (int)v[1], (int)v[2], F, (int)v[4], v[3], nullptr, F, v[3], nullptr,
                                     (int)v[3], (int32_t*)F, (int32_t*)F, F, (size_t)-1, nullptr);
        else if (op == "unsort")
            status = seedmm_moe_unsort(F, (int)v[3], v[2], (int)(v[0] * v[1]), (int32_t*)F, nullptr, F, (int)v[4], v[2], (int)v[0],
                                       (int)v[1], (int)v[2], nullptr);
        else if (op == "grad")
            status = seedmm_moe_unsort_grad(F, (int)v[3], v[2], F, (int)v[4], v[2], (int)(v[0] * v[1]), (int32_t*)F, (float*)F,
                                            F + 0x100000, v[2], (float*)F, (int)v[0], (int)v[1], (int)v[2], nullptr);
        else if (op == "swiglu")
            status = seedmm_swiglu(F, (int)v[2], 2 * v[1], F, (int)v[3], v[1], v[3] == SEEDMM_I8 ? (float*)F : nullptr, nullptr,
                                   (int)v[0], (int)v[1], nullptr);
        else
            status = -1;
        if (status != SEEDMM_OK) {
            std::cerr << "status " << status << " of: " << line << "\n";
            return 1;
        }
        std::cout << launched << "\n";
    }
    return 0;
}
