// Prints what the library's rules say on 256 CUs: a line "own T WORKGROUPS" of its input asks
// whether the experts' workgroups choose for themselves, "few M N" whether the INT8 product of M
// rows and N outputs takes the kernel for few rows.
#include <cstdint>
#include <cstdio>
#include <cstring>

namespace convrot {
bool moe_own_choice(int T, int64_t workgroups, int64_t cus);
bool few_rows(int64_t M, int64_t N, int64_t cus);
} // namespace convrot

int main()
{
    char rule[16];
    long long a, b;
    while (std::scanf("%15s %lld %lld", rule, &a, &b) == 3)
        if (!std::strcmp(rule, "own")) std::printf("%d\n", convrot::moe_own_choice((int)a, b, 256));
        else if (!std::strcmp(rule, "few")) std::printf("%d\n", convrot::few_rows(a, b, 256));
        else return 1;
}
